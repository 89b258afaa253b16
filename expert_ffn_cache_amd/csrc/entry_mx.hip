// Whole (layer, expert) entries between bf16 / fp32 and MXFP4.
//
// Conversion of a block V of 32 contraction elements (the MX rule): s = floor(log2 max |V|) - 2
// + 127, at least 0; each element is V / 2^(s - 127) rounded to nearest on the E2M1 grid, ties
// to the even code, magnitudes beyond 6 saturating to 6 (which is what
// v_cvt_scalef32_pk_fp4_{f32,bf16} does).  A block that holds an infinity or a NaN gets the
// scale 255 and dequantises to NaN.
//
// Work split: a thread owns one block (64 bytes of bf16, 128 of fp32; 16 code bytes and a scale
// byte).  Blocks are numbered as the MXFP4 entry stores them (inside a 16-row strip: block b of
// all 16 rows, then block b + 1), so the code side is contiguous over a wave and the other side
// covers 16 rows x 256 (512) bytes.  HBM-bound: 2.53 (4.53) bytes a weight.
#include <algorithm>

#include "mx8_dev.h"

using namespace moe;

namespace {

// Block g of an entry (numbered over the three matrices in storage order): its first element
// in the plain layout, its 16 code bytes and its scale byte in the MXFP4 layout.
struct BlockAt {
  size_t elem, code, scale;
};
__device__ __forceinline__ BlockAt block_at(unsigned g, unsigned per_mat, int d, int f) {
  const unsigned m = g / per_mat, b = g - m * per_mat;  // matrix, block in the matrix
  const unsigned K = m == 2 ? f : d, per_strip = K >> 1;  // 16 rows x K/32 blocks
  const unsigned rt = b / per_strip, in = b - rt * per_strip;
  const unsigned row = rt * 16 + (in & 15), kb = in >> 4;
  return BlockAt{(size_t)m * d * f + (size_t)row * K + kb * 32, (size_t)g * 16,
                 3 * ((size_t)d * f / 2) + g};
}

template <int SDT>
__global__ __launch_bounds__(256) void entry_quantize(const char* src, size_t src_stride, int d,
                                                      int f, char* dst, size_t dst_stride) {
  const unsigned per_mat = (unsigned)((size_t)d * f / 32);
  const char* se = src + blockIdx.y * src_stride;
  char* de = dst + blockIdx.y * dst_stride;
  for (unsigned g = blockIdx.x * 256 + threadIdx.x; g < 3 * per_mat; g += gridDim.x * 256) {
    const BlockAt at = block_at(g, per_mat, d, f);
    u32x4 v[SDT == MOE_F32 ? 8 : 4];
    const char* s = se + at.elem * (SDT == MOE_F32 ? 4 : 2);
#pragma unroll
    for (int i = 0; i < (SDT == MOE_F32 ? 8 : 4); ++i) v[i] = ldg16(s + 16 * i);
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < (SDT == MOE_F32 ? 8 : 4); ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if (SDT == MOE_F32) m = max(m, v[i][q] & 0x7FFFFFFFu);
        else m = max(m, max(v[i][q] & 0x7FFF0000u, (v[i][q] << 16) & 0x7FFF0000u));
      }
    const int e = (int)(m >> 23);
    const uint32_t sb = e == 255 ? 255u : (uint32_t)max(e - 2, 0);
    u32x4 c{0u, 0u, 0u, 0u};
    if (e != 255) {
      const float sc = e8m0_value(sb);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t w = 0;
        if (SDT == MOE_F32) {
          const f32x4 a = __builtin_bit_cast(f32x4, v[2 * i]), b = __builtin_bit_cast(f32x4, v[2 * i + 1]);
          w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, a[0], a[1], sc, 0);
          w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, a[2], a[3], sc, 1);
          w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, b[0], b[1], sc, 2);
          w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, b[2], b[3], sc, 3);
        } else {
          const uint32_t p0 = v[i][0], p1 = v[i][1], p2 = v[i][2], p3 = v[i][3];
          w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(bf16x2, p0), sc, 0);
          w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(bf16x2, p1), sc, 1);
          w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(bf16x2, p2), sc, 2);
          w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(bf16x2, p3), sc, 3);
        }
        c[i] = w;
      }
    }
    *(u32x4*)(de + at.code) = c;
    de[at.scale] = (char)sb;
  }
}

template <int DDT>
__global__ __launch_bounds__(256) void entry_dequantize(const char* src, size_t src_stride, int d,
                                                        int f, char* dst, size_t dst_stride) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  const unsigned per_mat = (unsigned)((size_t)d * f / 32);
  const char* se = src + blockIdx.y * src_stride;
  char* de = dst + blockIdx.y * dst_stride;
  for (unsigned g = blockIdx.x * 256 + threadIdx.x; g < 3 * per_mat; g += gridDim.x * 256) {
    const BlockAt at = block_at(g, per_mat, d, f);
    const u32x4 c = ldg16(se + at.code);
    const uint32_t sb = ldg_u8(se + at.scale);
    const bool nan = sb == 255u;
    const float sc = e8m0_value(sb);
    char* o = de + at.elem * (DDT == MOE_F32 ? 4 : 2);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (DDT == MOE_F32) {
        const f32x2 v0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[i], sc, 0);
        const f32x2 v1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[i], sc, 1);
        const f32x2 v2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[i], sc, 2);
        const f32x2 v3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[i], sc, 3);
        const float q = __uint_as_float(0x7FC00000u);
        *(f32x4*)(o + 32 * i) = nan ? f32x4{q, q, q, q} : f32x4{v0[0], v0[1], v1[0], v1[1]};
        *(f32x4*)(o + 32 * i + 16) = nan ? f32x4{q, q, q, q} : f32x4{v2[0], v2[1], v3[0], v3[1]};
      } else {
        const u32x4 w{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c[i], sc, 0)),
                      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c[i], sc, 1)),
                      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c[i], sc, 2)),
                      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c[i], sc, 3))};
        const uint32_t q = 0x7FC07FC0u;
        *(u32x4*)(o + 16 * i) = nan ? u32x4{q, q, q, q} : w;
      }
    }
  }
}

int entry_check(int n, int d, int f, int dt, size_t plain_stride, size_t mx_stride) {
  if (n < 0 || d <= 0 || f <= 0 || d % 64 != 0 || f % 64 != 0) return MOE_EINVAL;
  if ((size_t)d * f > (size_t)1 << 35) return MOE_EINVAL;  // block numbers are 32-bit
  if (dt != MOE_F32 && dt != MOE_BF16) return MOE_EUNSUPPORTED;
  if (plain_stride % 16 != 0 || mx_stride % 16 != 0) return MOE_EINVAL;
  if (plain_stride < moe_entry_bytes(d, f, dt) || mx_stride < moe_entry_bytes(d, f, MOE_MXFP4)) return MOE_EINVAL;
  return MOE_OK;
}

// Entries are a grid dimension of their own, at most 65535 of them a launch.
constexpr int kEntriesPerLaunch = 65535;
dim3 entry_grid(int n, int d, int f) {
  const size_t blocks = 3 * ((size_t)d * f / 32);
  return dim3((unsigned)std::min<size_t>((blocks + 255) / 256, 1 << 15), (unsigned)std::min(n, kEntriesPerLaunch));
}

}  // namespace

extern "C" int moe_entry_quantize(const void* src, int src_dtype, size_t src_stride, int n, int d,
                                  int f, void* dst, size_t dst_stride, hipStream_t stream) {
  if (int rc = entry_check(n, d, f, src_dtype, src_stride, dst_stride)) return rc;
  if (n == 0) return MOE_OK;
  if (!src || !dst || !moe_aligned16(src) || !moe_aligned16(dst)) return MOE_EINVAL;
  for (int i = 0; i < n; i += kEntriesPerLaunch) {
    const dim3 grid = entry_grid(n - i, d, f);
    const char* s = (const char*)src + i * src_stride;
    char* o = (char*)dst + i * dst_stride;
    if (src_dtype == MOE_F32) hipLaunchKernelGGL(entry_quantize<MOE_F32>, grid, dim3(256), 0, stream, s, src_stride, d, f, o, dst_stride);
    else hipLaunchKernelGGL(entry_quantize<MOE_BF16>, grid, dim3(256), 0, stream, s, src_stride, d, f, o, dst_stride);
    MOE_LAUNCH_CHECK();
  }
  return MOE_OK;
}

extern "C" int moe_entry_dequantize(const void* src, size_t src_stride, int n, int d, int f,
                                    void* dst, int dst_dtype, size_t dst_stride, hipStream_t stream) {
  if (int rc = entry_check(n, d, f, dst_dtype, dst_stride, src_stride)) return rc;
  if (n == 0) return MOE_OK;
  if (!src || !dst || !moe_aligned16(src) || !moe_aligned16(dst)) return MOE_EINVAL;
  for (int i = 0; i < n; i += kEntriesPerLaunch) {
    const dim3 grid = entry_grid(n - i, d, f);
    const char* s = (const char*)src + i * src_stride;
    char* o = (char*)dst + i * dst_stride;
    if (dst_dtype == MOE_F32) hipLaunchKernelGGL(entry_dequantize<MOE_F32>, grid, dim3(256), 0, stream, s, src_stride, d, f, o, dst_stride);
    else hipLaunchKernelGGL(entry_dequantize<MOE_BF16>, grid, dim3(256), 0, stream, s, src_stride, d, f, o, dst_stride);
    MOE_LAUNCH_CHECK();
  }
  return MOE_OK;
}
