// The 8-bit activation checkpoints of rows: r2l_act8_pack and r2l_act8_unpack.
//
// Both move bytes and little else (pack reads 2 or 4 bytes a value and writes
// 1, unpack the reverse), so what counts is wide accesses in flight: a warp
// takes 4 rows of 256 channels, their loads first.  Rows on 16-byte boundaries
// give a lane 8 channels of a row, 8 lanes a group; others are read element by
// element, 32 neighbours at a time.  8 x 4096 rows of 2048 in bf16: pack 38 us
// (5.3 TB/s), unpack 33 us (6.1 TB/s); of 8 x 2048 x 1037, whose rows start
// anywhere, 51 and 22 us (1.0 and 2.3 TB/s).  Infinities, NaN and values that
// would round to 2^128 are looked for only where a group's largest bits say that
// there is one.
#include "act8.cuh"
#include "gated_host.cuh"

using namespace r2l::gated;
using r2l::bf16;
using r2l::from_f32;
using r2l::to_f32;
using r2l::act8::GROUP;

namespace {

constexpr int WROWS = 4, WCOLS = 256, WARPS = 8;    // rows and channels of a warp, warps of a block
constexpr int WGROUPS = WCOLS / GROUP;

// The rows of a warp: m0 … m0 + 3 of the batch, as bits the valid ones.
struct Rows {
  long long m0;
  int col0;
  uint32_t valid;
};
__device__ __forceinline__ Rows my_rows(int B, int L, int cols, const int32_t* lengths) {
  const unsigned blocks = (cols + WCOLS - 1) / WCOLS;
  Rows r;
  r.col0 = (int)(blockIdx.x % blocks) * WCOLS;
  r.m0 = ((long long)(blockIdx.x / blocks) * WARPS + (threadIdx.x >> 5)) * WROWS;
  long long b = r.m0 / L;
  int i = (int)(r.m0 - b * L);
  r.valid = 0;
#pragma unroll
  for (int j = 0; j < WROWS; ++j) {
    if (b < B && i < clamped_length(lengths, (int)b, L)) r.valid |= 1u << j;
    if (++i == L) i = 0, ++b;
  }
  return r;
}

// 8 channels of a lane.
struct Eight {
  float v[8];
};
__device__ __forceinline__ void load8(const bf16* p, uint4* raw) { raw[0] = *reinterpret_cast<const uint4*>(p); }
__device__ __forceinline__ void load8(const float* p, uint4* raw) {
  raw[0] = reinterpret_cast<const uint4*>(p)[0];
  raw[1] = reinterpret_cast<const uint4*>(p)[1];
}
__device__ __forceinline__ Eight widen(const uint4* raw, bf16) {
  const uint32_t w[4] = {raw[0].x, raw[0].y, raw[0].z, raw[0].w};
  Eight e;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    e.v[2 * k] = __uint_as_float(w[k] << 16);
    e.v[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
  }
  return e;
}
__device__ __forceinline__ Eight widen(const uint4* raw, float) {
  Eight e;
  *reinterpret_cast<uint4*>(e.v) = raw[0];
  *reinterpret_cast<uint4*>(e.v + 4) = raw[1];
  return e;
}
__device__ __forceinline__ void store8(bf16* p, const Eight& e) {
  uint4 w;
  uint32_t* u = &w.x;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const __nv_bfloat162 two = __floats2bfloat162_rn(e.v[2 * k], e.v[2 * k + 1]);
    u[k] = *reinterpret_cast<const uint32_t*>(&two);
  }
  *reinterpret_cast<uint4*>(p) = w;
}
__device__ __forceinline__ void store8(float* p, const Eight& e) {
  reinterpret_cast<float4*>(p)[0] = make_float4(e.v[0], e.v[1], e.v[2], e.v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(e.v[4], e.v[5], e.v[6], e.v[7]);
}

template <typename T>
__global__ void __launch_bounds__(WARPS * 32) act8_pack_wide_kernel(const T* x, long long ldx, int B, int L, int cols,
                                                                    const int32_t* lengths, uint8_t* q, long long ldq,
                                                                    uint8_t* scales) {
  const Rows r = my_rows(B, L, cols, lengths);
  const int lane = threadIdx.x & 31, c = r.col0 + lane * 8, groups = (cols + GROUP - 1) / GROUP;
  const bool in = c < cols;      // cols is a multiple of 8
  uint4 raw[WROWS][sizeof(T) / 2];
#pragma unroll
  for (int j = 0; j < WROWS; ++j)
    if (in && (r.valid >> j & 1)) load8(x + (r.m0 + j) * ldx + c, raw[j]);
#pragma unroll
  for (int j = 0; j < WROWS; ++j) {
    const bool on = in && (r.valid >> j & 1);
    Eight e{};
    if (on) e = widen(raw[j], T());
    uint32_t top = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) top = max(top, __float_as_uint(e.v[k]) & 0x7fffffffu);
#pragma unroll
    for (int d = 1; d < 8; d *= 2) top = max(top, __shfl_xor_sync(0xffffffffu, top, d));
    const bool odd = __any_sync(0xffffffffu, top >= r2l::act8::SPECIAL);
    if (odd) {     // an infinity or a NaN does not count for the scale
      top = 0;
      for (int k = 0; k < 8; ++k) {
        top = max(top, r2l::act8::finite_abs_bits(e.v[k]));
        e.v[k] = r2l::act8::storable(e.v[k]);
      }
      for (int d = 1; d < 8; d *= 2) top = max(top, __shfl_xor_sync(0xffffffffu, top, d));
    }
    if (!on) continue;
    const uint32_t byte = r2l::act8::scale_byte(top);
    const float down = r2l::act8::scale_down(byte);
    uint32_t w[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      float s[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) s[i] = e.v[4 * k + i] * down;
      w[k] = r2l::act8::to_e4m3x2(s[0], s[1]) | (uint32_t)r2l::act8::to_e4m3x2(s[2], s[3]) << 16;
    }
    *reinterpret_cast<uint2*>(q + (r.m0 + j) * ldq + c) = make_uint2(w[0], w[1]);
    if (lane % 8 == 0) scales[(r.m0 + j) * groups + c / GROUP] = (uint8_t)byte;
  }
}

template <typename T>
__global__ void __launch_bounds__(WARPS * 32) act8_pack_kernel(const T* x, long long ldx, int B, int L, int cols,
                                                               const int32_t* lengths, uint8_t* q, long long ldq,
                                                               uint8_t* scales) {
  const Rows r = my_rows(B, L, cols, lengths);
  const int lane = threadIdx.x & 31, c = r.col0 + lane, groups = (cols + GROUP - 1) / GROUP;
  float v[WROWS][WCOLS / 32];
#pragma unroll
  for (int j = 0; j < WROWS; ++j)
#pragma unroll
    for (int k = 0; k < WCOLS / 32; ++k)
      v[j][k] = (r.valid >> j & 1) && c + 32 * k < cols ? to_f32(x[(r.m0 + j) * ldx + c + 32 * k]) : 0.0f;
#pragma unroll
  for (int j = 0; j < WROWS; ++j) {
    if (!(r.valid >> j & 1)) continue;
#pragma unroll
    for (int g = 0; g < WGROUPS; ++g) {
      float a = v[j][2 * g], b = v[j][2 * g + 1];
      uint32_t top = __reduce_max_sync(0xffffffffu, max(__float_as_uint(a) & 0x7fffffffu, __float_as_uint(b) & 0x7fffffffu));
      if (top >= r2l::act8::SPECIAL) {     // an infinity or a NaN does not count for the scale
        top = __reduce_max_sync(0xffffffffu, max(r2l::act8::finite_abs_bits(a), r2l::act8::finite_abs_bits(b)));
        a = r2l::act8::storable(a);
        b = r2l::act8::storable(b);
      }
      const uint32_t byte = r2l::act8::scale_byte(top);
      const float down = r2l::act8::scale_down(byte);
      const uint16_t two = r2l::act8::to_e4m3x2(a * down, b * down);
      uint8_t* const to = q + (r.m0 + j) * ldq + c + 64 * g;
      if (c + 64 * g < cols) to[0] = (uint8_t)two;
      if (c + 64 * g + 32 < cols) to[32] = (uint8_t)(two >> 8);
      if (lane == 0 && r.col0 / GROUP + g < groups) scales[(r.m0 + j) * groups + r.col0 / GROUP + g] = (uint8_t)byte;
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(WARPS * 32) act8_unpack_wide_kernel(const uint8_t* q, long long ldq, const uint8_t* scales,
                                                                      int B, int L, int cols, const int32_t* lengths, T* out,
                                                                      long long ldo) {
  const Rows r = my_rows(B, L, cols, lengths);
  const int c = r.col0 + (threadIdx.x & 31) * 8, groups = (cols + GROUP - 1) / GROUP;
  if (c >= cols) return;
  uint2 raw[WROWS];
  uint32_t byte[WROWS];
#pragma unroll
  for (int j = 0; j < WROWS; ++j)
    if (r.valid >> j & 1) {
      raw[j] = *reinterpret_cast<const uint2*>(q + (r.m0 + j) * ldq + c);
      byte[j] = scales[(r.m0 + j) * groups + c / GROUP];
    }
#pragma unroll
  for (int j = 0; j < WROWS; ++j) {
    if (!(r.valid >> j & 1)) continue;
    const float up = r2l::act8::scale_up(byte[j]);
    Eight e;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t w = k < 2 ? raw[j].x : raw[j].y;
      const float2 v = r2l::act8::from_e4m3x2((uint16_t)(w >> (16 * (k % 2))));
      e.v[2 * k] = v.x * up;
      e.v[2 * k + 1] = v.y * up;
    }
    store8(out + (r.m0 + j) * ldo + c, e);
  }
}

template <typename T>
__global__ void __launch_bounds__(WARPS * 32) act8_unpack_kernel(const uint8_t* q, long long ldq, const uint8_t* scales, int B,
                                                                 int L, int cols, const int32_t* lengths, T* out,
                                                                 long long ldo) {
  const Rows r = my_rows(B, L, cols, lengths);
  const int c = r.col0 + (threadIdx.x & 31), groups = (cols + GROUP - 1) / GROUP;
#pragma unroll
  for (int j = 0; j < WROWS; ++j) {
    if (!(r.valid >> j & 1)) continue;
    uint8_t v[WCOLS / 32];
    uint32_t byte[WGROUPS];
#pragma unroll
    for (int k = 0; k < WCOLS / 32; ++k)
      if (c + 32 * k < cols) v[k] = q[(r.m0 + j) * ldq + c + 32 * k];
#pragma unroll
    for (int g = 0; g < WGROUPS; ++g)
      if (r.col0 / GROUP + g < groups) byte[g] = scales[(r.m0 + j) * groups + r.col0 / GROUP + g];
#pragma unroll
    for (int k = 0; k < WCOLS / 32; ++k)
      if (c + 32 * k < cols)
        out[(r.m0 + j) * ldo + c + 32 * k] =
            from_f32<T>(r2l::act8::from_e4m3x2(v[k]).x * r2l::act8::scale_up(byte[k / 2]));
  }
}

long long grid_of(int B, int L, int cols) {
  const long long rows = ((long long)B * L + WARPS * WROWS - 1) / (WARPS * WROWS);
  return rows * ((cols + WCOLS - 1LL) / WCOLS);
}

// Whether a lane may take 8 channels at once: of rows of T, and of the bytes.
bool wide(const void* rows, int ld, size_t size, const void* q, int ldq, int cols) {
  return rows16(rows, ld, size) && aligned(q, 8) && ldq % 8 == 0 && cols % 8 == 0;
}

r2l_status check(const void* rows, int ld, r2l_dtype dtype, int B, int L, int cols, const int32_t* lengths, const uint8_t* q,
                 int ldq, const uint8_t* scales) {
  if (B <= 0 || L <= 0 || cols <= 0 || (dtype != R2L_BF16 && dtype != R2L_FP32) || !scales) return R2L_ERR_INVALID_ARG;
  R2L_TRY(check_rows(rows, ld, cols, elem_bytes(dtype)));
  R2L_TRY(check_rows(q, ldq, cols, 1));
  if (rows == q || rows == scales || q == scales) return R2L_ERR_INVALID_ARG;
  if (!aligned(lengths, 4)) return R2L_ERR_ALIGNMENT;
  return fits(B, L, cols) && grid_of(B, L, cols) <= 2147483647LL ? R2L_OK : R2L_ERR_UNSUPPORTED;
}

}  // namespace

extern "C" {

r2l_status r2l_act8_pack(const void* x, int ldx, r2l_dtype dtype, int B, int L, int cols, const int32_t* lengths,
                         uint8_t* q, int ldq, uint8_t* scales, void* stream) {
  R2L_TRY(check(x, ldx, dtype, B, L, cols, lengths, q, ldq, scales));
  const unsigned grid = (unsigned)grid_of(B, L, cols);
  const cudaStream_t st = (cudaStream_t)stream;
  const bool w = wide(x, ldx, elem_bytes(dtype), q, ldq, cols);
  if (dtype == R2L_BF16)
    (w ? act8_pack_wide_kernel<bf16> : act8_pack_kernel<bf16>)<<<grid, WARPS * 32, 0, st>>>(
        (const bf16*)x, ldx, B, L, cols, lengths, q, ldq, scales);
  else
    (w ? act8_pack_wide_kernel<float> : act8_pack_kernel<float>)<<<grid, WARPS * 32, 0, st>>>(
        (const float*)x, ldx, B, L, cols, lengths, q, ldq, scales);
  R2L_LAUNCH_CHECK();
  return R2L_OK;
}

r2l_status r2l_act8_unpack(const uint8_t* q, int ldq, const uint8_t* scales, r2l_dtype dtype, int B, int L, int cols,
                           const int32_t* lengths, void* out, int ldo, void* stream) {
  R2L_TRY(check(out, ldo, dtype, B, L, cols, lengths, q, ldq, scales));
  const unsigned grid = (unsigned)grid_of(B, L, cols);
  const cudaStream_t st = (cudaStream_t)stream;
  const bool w = wide(out, ldo, elem_bytes(dtype), q, ldq, cols);
  if (dtype == R2L_BF16)
    (w ? act8_unpack_wide_kernel<bf16> : act8_unpack_kernel<bf16>)<<<grid, WARPS * 32, 0, st>>>(
        q, ldq, scales, B, L, cols, lengths, (bf16*)out, ldo);
  else
    (w ? act8_unpack_wide_kernel<float> : act8_unpack_kernel<float>)<<<grid, WARPS * 32, 0, st>>>(
        q, ldq, scales, B, L, cols, lengths, (float*)out, ldo);
  R2L_LAUNCH_CHECK();
  return R2L_OK;
}

}  // extern "C"
