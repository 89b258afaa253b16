// Expert FFN with MXFP8 activations and MXFP4 weights, weight-streaming form (few rows per
// expert): both operands go to the block-scaled matrix instruction as they are stored,
//   v_mfma_scale_f32_16x16x128_f8f6f4:  D += (A 2^(sA - 127)) (B 2^(sB - 127))^T,
// with one scale per operand row and 32 reduction elements and fp32 accumulation, so no code
// is expanded and the kernels do nothing but stream the weights.
//
// A = weights: a tile of the entry layout (16 rows x 128 elements, slot 16 q + i = row i,
// elements 32 q .. 32 q + 31) is exactly the operand: lane 16 q + i holds row i, reduction block
// q, 16 code bytes and that block's scale.  B = token rows (E4M3): lane 16 q + i holds token i,
// bytes 16 q .. 16 q + 15 and 64 + 16 q .. 64 + 16 q + 15 of the tile's 128 (the instruction's
// order for 8-bit operands), and the scale of block q.  D: lane 16 g + i holds weight rows
// 4 g .. 4 g + 3 of token i.
//
// h is rounded to MXFP8 too (blocks of 32 units), so a wave takes two adjacent 16-row strips
// of both gate and up: a block of h is then 8 values in each of four lanes, and its scale takes
// two lane exchanges.  A workgroup's four waves take four strip pairs of one expert, or (KS = 2,
// 4, when the strips are too few to fill the chip) share them, tiles ks, ks + KS, ..., their
// partial sums meeting in LDS.
//
// Token rows (at most 16 per pass; experts with more rows make several passes) are staged in
// LDS over a slice of the contraction that fits 32 KB: 8192 elements for up to 4 rows, 4096 for
// 8, 2048 for 16; the accumulators carry over from slice to slice.
#include <algorithm>

#include "mx8_dev.h"
#include "mx_dev.h"

namespace moe {
namespace {

constexpr int kM8Ahead = 2;              // weight tiles in flight per wave and matrix
constexpr int kM8Codes = 32768;          // LDS bytes of staged codes
constexpr int kM8Pad = 16;               // bytes between staged rows (bank spread)

// A workgroup's expert, its rows and its entry: the a-th active expert in ascending id, found by
// every wave for itself (the same cached offsets; no barrier), 256 experts a round trip; n = 0 past
// the last or without an entry.
struct M8Item {
  int n0, n;
  const uint8_t* w;
};
__device__ __forceinline__ M8Item m8_item(const FfnArgs& p, int a) {
  const int lane = threadIdx.x & 63;
  int seen = 0;
  for (int e0 = 0; e0 < p.E; e0 += 256) {
    int lo[4], hi[4];
    bool on[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int e = min(e0 + 64 * j + lane, p.E - 1);
      lo[j] = p.offsets[e];
      hi[j] = p.offsets[e + 1];
      on[j] = !p.mask || p.mask[e];
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int n = hi[j] - lo[j];
      const bool act = e0 + 64 * j + lane < p.E && n > 0 && n >= p.nmin && n <= p.nmax && on[j];
      const unsigned long long m = __ballot(act);
      const int c = __popcll(m);
      if (a < seen + c) {
        const bool mine = act && __popcll(m & lanemask_lt(lane)) == a - seen;
        const int l = __builtin_amdgcn_readfirstlane(__ffsll((long long)__ballot(mine)) - 1);
        const uint8_t* w = (const uint8_t*)entry_of(p, e0 + 64 * j + l);
        return M8Item{__builtin_amdgcn_readlane(lo[j], l), w ? __builtin_amdgcn_readlane(n, l) : 0, w};
      }
      seen += c;
    }
  }
  return M8Item{0, 0, nullptr};
}

__device__ __forceinline__ int m8_rows_class(int n) { return n <= 4 ? 4 : n <= 8 ? 8 : 16; }

// LDS of a workgroup: staged codes with their row padding, then the scales (4 per tile and row).
struct M8Lds {
  uint8_t codes[kM8Codes + 16 * kM8Pad];
  uint8_t scales[kM8Codes / 32];
};

// Tiles t0 .. t1 - 1 of nt rows into LDS: codes at row stride (t1 - t0) * 128 + pad, scales at
// 4 (t1 - t0).  Past K (a short last tile): zero codes and scale 2^0, so that the products
// with the zero weights there are zero.
template <typename RowOf>
__device__ __forceinline__ void m8_stage(M8Lds& lds, const uint8_t* codes, const uint8_t* scales,
                                         int K, int t0, int t1, int nt, RowOf src_row) {
  const int ss = mxfp8_scale_stride(K), nch = (t1 - t0) * 8, stride = (t1 - t0) * 128 + kM8Pad;
  __syncthreads();  // the previous slice's readers are done
  for (int c = threadIdx.x; c < nt * nch; c += 256) {
    const int t = c / nch, b = c - t * nch, k = t0 * 128 + b * 16;
    *(u32x4*)&lds.codes[t * stride + b * 16] = k < K ? ldg16(codes + (size_t)src_row(t) * K + k) : u32x4{0u, 0u, 0u, 0u};
  }
  for (int c = threadIdx.x; c < nt * (t1 - t0); c += 256) {
    const int t = c / (t1 - t0), b = c - t * (t1 - t0);
    uint32_t s = *(const uint32_t*)(scales + (size_t)src_row(t) * ss + (t0 + b) * 4);
    if ((t0 + b) * 128 + 64 >= K) s = (s & 0xFFFFu) | 0x7F7F0000u;
    *(uint32_t*)&lds.scales[c * 4] = s;
  }
  __syncthreads();
}

template <int NMAT>
__device__ __forceinline__ void m8_tile_mma(const MxTile<NMAT>& t, const uint8_t* x, uint32_t xs,
                                            f32x4 (&acc)[NMAT]) {
  const i32x8 b = fp8_operand(*(const u32x4*)x, *(const u32x4*)(x + 64));
#pragma unroll
  for (int m = 0; m < NMAT; ++m)
    acc[m] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fp4_operand(t.c[m]), b, acc[m], 4, 0, 0,
                                                              (int)t.s[m], 0, (int)xs);
}

// Partial sums of the KS waves of each strip pair, through the staged rows' LDS: waves ks > 0
// store, then the first wave adds.
template <int NMAT, int KS>
__device__ __forceinline__ void m8_reduce(M8Lds& lds, f32x4 (&acc)[NMAT], int pr, int ks, int lane) {
  if (KS == 1) return;
  f32x4* red = (f32x4*)lds.codes;  // [3][NMAT][64]
  __syncthreads();  // the staged rows are read
  if (ks > 0) {
#pragma unroll
    for (int m = 0; m < NMAT; ++m) red[((pr * (KS - 1) + ks - 1) * NMAT + m) * 64 + lane] = acc[m];
  }
  __syncthreads();
  if (ks == 0) {
#pragma unroll
    for (int j = 1; j < KS; ++j)
#pragma unroll
      for (int m = 0; m < NMAT; ++m) acc[m] += red[((pr * (KS - 1) + j - 1) * NMAT + m) * 64 + lane];
  }
}

// The wave's share of all K for one block of up to 16 rows: acc[m] (+)= strip m x rows.
template <int NMAT, int KS, typename RowOf>
__device__ __forceinline__ void m8_rows(M8Lds& lds, const uint8_t* codes, const uint8_t* scales,
                                        int K, int nt, RowOf src_row, const uint8_t* const (&cb)[NMAT],
                                        const uint8_t* const (&sb)[NMAT], int ks, int lane, bool work,
                                        f32x4 (&acc)[NMAT]) {
  const int nk = (K + 127) >> 7, q = lane >> 4, col = min(lane & 15, nt - 1);
  const int tps = min(nk, 256 / m8_rows_class(nt));
  const int kshort = (K & 127) ? nk - 1 : -1;
#pragma unroll
  for (int m = 0; m < NMAT; ++m) acc[m] = f32x4{0.f, 0.f, 0.f, 0.f};
  for (int t0 = 0; t0 < nk; t0 += tps) {
    const int t1 = min(nk, t0 + tps);
    const int ntw = work && t1 - t0 > ks ? (t1 - t0 - ks + KS - 1) / KS : 0;  // tiles of this wave
    MxTile<NMAT> ring[kM8Ahead];
#pragma unroll
    for (int r = 0; r < kM8Ahead; ++r) {
      const int kt = t0 + ks + KS * r;
      if (r < ntw) mx_load_tile<NMAT>(ring[r], cb, sb, kt, lane, kt != kshort || q < 2);
    }
    m8_stage(lds, codes, scales, K, t0, t1, nt, src_row);
    const uint8_t* xr = lds.codes + col * ((t1 - t0) * 128 + kM8Pad) + 16 * q;
    const uint8_t* sr = lds.scales + col * (t1 - t0) * 4 + q;
    for (int i = 0; i < ntw; i += kM8Ahead) {
#pragma unroll
      for (int r = 0; r < kM8Ahead; ++r) {
        if (i + r < ntw) {
          const int kt = t0 + ks + KS * (i + r);
          m8_tile_mma<NMAT>(ring[r], xr + (kt - t0) * 128, sr[(kt - t0) * 4], acc);
          const int kn = kt + KS * kM8Ahead;
          if (i + r + kM8Ahead < ntw) mx_load_tile<NMAT>(ring[r], cb, sb, kn, lane, kn != kshort || q < 2);
        }
      }
    }
  }
}

// Four lanes 16 g + i hold 8 units each of token i's 32-unit block of h (strip 0: units 4 g ..
// 4 g + 3, strip 1: 16 + 4 g ..): converts them and writes the codes and the scale.
__device__ __forceinline__ void m8_store_h(uint8_t* codes, uint8_t* scale, int lane,
                                           const float (&h)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, abs_bits(h[i]));
  m = max(m, (uint32_t)__shfl_xor((int)m, 16));
  m = max(m, (uint32_t)__shfl_xor((int)m, 32));
  const uint32_t s = mxfp8_scale_of(m);
  const float sc = e8m0_value(s);
  const int g = lane >> 4;
  const uint32_t lo = mxfp8_pack4(h[0], h[1], h[2], h[3], s, sc), hi = mxfp8_pack4(h[4], h[5], h[6], h[7], s, sc);
  if (codes) {
    *(uint32_t*)(codes + 4 * g) = lo;
    *(uint32_t*)(codes + 16 + 4 * g) = hi;
    if (g == 0) *scale = (uint8_t)s;
  }
}

// Gate/up: workgroup = 4/KS pairs of strips (32 units each) of one expert.
template <int KS>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(4))) void m8_gateup(FfnArgs p, const uint8_t* xs, uint8_t* hs) {
  __shared__ __attribute__((aligned(16))) M8Lds lds;
  constexpr int TR = 4 / KS;
  const int npair = p.f >> 5, nb = (npair + TR - 1) / TR;
  const int a = blockIdx.x / nb, sb0 = blockIdx.x - a * nb;
  const M8Item it = m8_item(p, a);
  const int n0 = it.n0, n = it.n;
  if (!n) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int pr = wave / KS, ks = wave - pr * KS, pair = sb0 * TR + pr;
  const bool work = pair < npair;
  const int K = p.d;
  const size_t fd = (size_t)p.f * K, so = (size_t)(work ? pair : 0) * 16 * K, sso = (size_t)(work ? pair : 0) * K;
  const uint8_t* W = it.w;
  const uint8_t* S = W + 3 * (fd / 2);
  const uint8_t* const cb[4] = {W + so, W + so + 8 * (size_t)K, W + fd / 2 + so, W + fd / 2 + so + 8 * (size_t)K};
  const uint8_t* const sb[4] = {S + sso, S + sso + K / 2, S + fd / 32 + sso, S + fd / 32 + sso + K / 2};
  const int hss = mxfp8_scale_stride(p.f);
  for (int m0 = 0; m0 < n; m0 += 16) {
    const int nt = min(16, n - m0);
    f32x4 acc[4];
    m8_rows<4, KS>(lds, (const uint8_t*)p.x, xs, K, nt, [&](int t) { return p.perm[n0 + m0 + t] / p.k; }, cb, sb,
                   ks, lane, work, acc);
    m8_reduce<4, KS>(lds, acc, pr, ks, lane);
    if (ks == 0 && work) {
      float h[8];
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int i = 0; i < 4; ++i) h[4 * s + i] = silu(acc[s][i]) * acc[2 + s][i];
      const int t = lane & 15;
      const size_t row = (size_t)(n0 + m0 + t);
      m8_store_h(t < nt ? (uint8_t*)p.h + row * p.f + 32 * pair : nullptr, hs + row * hss + pair, lane, h);
    }
  }
}

// Down: workgroup = 4/KS pairs of strips (32 output channels each) of one expert.
template <int KS, int YDT>
__global__ __launch_bounds__(256) void m8_down(FfnArgs p, const uint8_t* hs) {
  __shared__ __attribute__((aligned(16))) M8Lds lds;
  constexpr int TR = 4 / KS;
  const int npair = p.d >> 5, nb = (npair + TR - 1) / TR;
  const int a = blockIdx.x / nb, sb0 = blockIdx.x - a * nb;
  const M8Item it = m8_item(p, a);
  const int n0 = it.n0, n = it.n;
  if (!n) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int pr = wave / KS, ks = wave - pr * KS, pair = sb0 * TR + pr;
  const bool work = pair < npair;
  const int K = p.f;
  const size_t fd = (size_t)K * p.d, so = (size_t)(work ? pair : 0) * 16 * K, sso = (size_t)(work ? pair : 0) * K;
  const uint8_t* W = it.w + fd;
  const uint8_t* S = it.w + 3 * (fd / 2) + 2 * (fd / 32);
  const uint8_t* const cb[2] = {W + so, W + so + 8 * (size_t)K};
  const uint8_t* const sb[2] = {S + sso, S + sso + K / 2};
  for (int m0 = 0; m0 < n; m0 += 16) {
    const int nt = min(16, n - m0);
    f32x4 acc[2];
    m8_rows<2, KS>(lds, (const uint8_t*)p.h, hs, K, nt, [&](int t) { return n0 + m0 + t; }, cb, sb, ks, lane, work, acc);
    m8_reduce<2, KS>(lds, acc, pr, ks, lane);
    const int t = lane & 15, g = lane >> 4;
    if (ks == 0 && work && t < nt) {
      const size_t o = (size_t)(n0 + m0 + t) * p.d + 32 * pair + 4 * g;
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        if (YDT == MOE_F32) {
          *(f32x4*)((float*)p.y + o + 16 * s) = acc[s];
        } else {
          *(u32x2*)((uint16_t*)p.y + o + 16 * s) =
              u32x2{(uint32_t)f32_to_bf16(acc[s][0]) | (uint32_t)f32_to_bf16(acc[s][1]) << 16,
                    (uint32_t)f32_to_bf16(acc[s][2]) | (uint32_t)f32_to_bf16(acc[s][3]) << 16};
        }
      }
    }
  }
}

// Waves per strip pair: one unless that leaves fewer than 4 workgroups per CU.
int m8_ks(int experts, int R) {
  const long pairs = (long)experts * (R / 32);
  return pairs / 4 >= 1024 ? 1 : pairs / 2 >= 1024 ? 2 : 4;
}

template <int KS>
void launch_gu(const FfnArgs& p, const uint8_t* xs, uint8_t* hs, int experts, hipStream_t stream) {
  const int nb = (p.f / 32 * KS + 3) / 4;
  hipLaunchKernelGGL(m8_gateup<KS>, dim3(experts * nb), dim3(256), 0, stream, p, xs, hs);
}
template <int KS>
void launch_dn(const FfnArgs& p, const uint8_t* hs, int y_dtype, int experts, hipStream_t stream) {
  const dim3 grid(experts * ((p.d / 32 * KS + 3) / 4));
  if (y_dtype == MOE_F32) hipLaunchKernelGGL((m8_down<KS, MOE_F32>), grid, dim3(256), 0, stream, p, hs);
  else hipLaunchKernelGGL((m8_down<KS, MOE_BF16>), grid, dim3(256), 0, stream, p, hs);
}

}  // namespace

int launch_ffn_mx8(const FfnArgs& p, int T, int y_dtype, hipStream_t stream, int experts) {
  if (experts <= 0) return MOE_OK;
  const uint8_t* xs = (const uint8_t*)p.x + (size_t)T * p.d;
  uint8_t* hs = (uint8_t*)p.h + (size_t)T * p.k * p.f;
  switch (m8_ks(experts, p.f)) {
    case 1: launch_gu<1>(p, xs, hs, experts, stream); break;
    case 2: launch_gu<2>(p, xs, hs, experts, stream); break;
    default: launch_gu<4>(p, xs, hs, experts, stream); break;
  }
  MOE_LAUNCH_CHECK();
  switch (m8_ks(experts, p.d)) {
    case 1: launch_dn<1>(p, hs, y_dtype, experts, stream); break;
    case 2: launch_dn<2>(p, hs, y_dtype, experts, stream); break;
    default: launch_dn<4>(p, hs, y_dtype, experts, stream); break;
  }
  MOE_LAUNCH_CHECK();
  return MOE_OK;
}

}  // namespace moe
