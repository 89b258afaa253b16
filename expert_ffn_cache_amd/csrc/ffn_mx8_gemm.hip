// Expert FFN with MXFP8 activations and MXFP4 weights for many rows per expert: a grouped GEMM on
// v_mfma_scale_f32_32x32x64_f8f6f4, codes and scales of both sides as they are stored.
//
// Tile: 256 weight rows x 128 token rows of one expert, 4 waves, two workgroups a CU; a wave
// computes 64 weight rows x up to 128 token rows (2 x 4 accumulator tiles).  A = weights, B = tokens, so a lane holds
// 16 of the 32 weight rows of one token (the other 16 are in the lane 32 away): in gate/up
// (tile 0 gate, tile 1 up of the same 32 units) a block of h is two lanes, and its MXFP8 scale
// takes one exchange.
//
// k steps of 128 elements (one tile column of the entry layout) go through an LDS ring by direct
// global-to-LDS loads.  Operand order of the instruction (lane 32 g + i, elements of the 64 in
// step half kh): FP4 row i: elements 32 g .. 32 g + 31, which is block 2 kh + g of the row and one
// 16-byte slot of the weight tile; E4M3 row i: 16 g .. and 32 + 16 g .., two 16-byte pieces; the
// scale of lane 32 g + i is that of row i, block 2 kh + g.  A token row's four scales of the step
// are one word, shifted so that the lane's two are bytes 0 and 2, which the instruction
// selects.  Token rows lie at 128 bytes with their 16-byte pieces permuted by (row / 2) mod 8
// (16 lanes that read one piece of 16 rows then touch all banks once).
//
// Work list: persistent workgroups over (expert, weight tile, token tile), derived from the
// offsets on the device; consecutive items, which share weights or token rows, go to one XCD.
// Token tiles go four at a time to a weight tile, so its codes come from L2 for three of them.
#include <algorithm>
#include <type_traits>

#include "mx8_dev.h"

namespace moe {
namespace {

constexpr int kGCodes = 16 * 1024;       // codes of a stage: strip s at s * 1024, slot 16 q + i
constexpr int kGScales = 16 * 64;        // weight scales of a stage: strip s at s * 64

constexpr int kGM = 256;                 // token rows of a tile
// A stage: weight scales, token rows (row r at r * 128), codes.
constexpr int kGTokAt = kGScales;
constexpr int kGCodeAt = kGTokAt + kGM * 128;
constexpr int kGStage = kGCodeAt + kGCodes;
constexpr int kGStages = 3;
constexpr int kGLoads = 8;  // loads of a wave per stage
// Token scales come in chunks of 4 steps, two of them in LDS: row r's word of step n of a chunk at
// word r * 4 + (n ^ (r / 16) mod 4).  One load brings 16 rows x 16 bytes; a word per row and step
// instead would fetch a whole cache line for it (that alone cost half of the time).
constexpr int kGTsWords = kGM * 4;

__device__ __forceinline__ uint32_t g_lds_addr(const void* p) {
  return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) void*)p;
}
// LDS reads at a byte address + a constant.
template <typename T>
__device__ __forceinline__ T g_lds(uint32_t at, int off) {
  return *(const __attribute__((address_space(3))) T*)(uintptr_t)(at + off);
}
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
// 64 lanes x 16 (4) bytes from base + the lane's offset to consecutive LDS bytes from `lds` on.
__device__ __forceinline__ void g_load16(const void* base, uint32_t off, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(lds), "v"(off), "s"(base) : "memory", "m0");
}
__device__ __forceinline__ void g_load4(const void* base, uint32_t off, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\tglobal_load_lds_dword %1, %2" ::"s"(lds), "v"(off), "s"(base) : "memory", "m0");
}
#pragma clang diagnostic pop
template <int N>
__device__ __forceinline__ void g_wait_loads() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(waitcnt_imm(N, 7, 15));
  asm volatile("" ::: "memory");
}

// SiLU(g) * u with the hardware reciprocal (1 ulp), as in the bf16 GEMMs.
__device__ __forceinline__ float g_swiglu(float g, float u) {
  return g * __builtin_amdgcn_rcpf(1.0f + __expf(-g)) * u;
}

// Words w[0..3] of lane 32 g + i are elements 8 j + 4 g .. of row i's 32 (4 bytes each or packed
// wider); afterwards lane 32 g + i holds words of elements 16 g .. 16 g + 15 in order.
__device__ __forceinline__ void g_pair_rows(uint32_t (&w)[4]) {
  const auto a = __builtin_amdgcn_permlane32_swap(w[0], w[2], false, false);
  const auto b = __builtin_amdgcn_permlane32_swap(w[1], w[3], false, false);
  w[0] = a[0]; w[1] = a[1]; w[2] = b[0]; w[3] = b[1];
}

template <int MODE, int YDT>  // MODE 0: gate/up (h out), 1: down (y out)
__global__ __launch_bounds__(512) __attribute__((amdgpu_waves_per_eu(2, 2)))
void m8_tile(FfnArgs p, const uint8_t* ascales, uint32_t last_piece, uint8_t* hscales, int n_ntiles) {
  __shared__ __attribute__((aligned(1024))) uint8_t sm[kGStages][kGStage];
  __shared__ int s_pref[kMaxE + 1];
  __shared__ int s_part[8];
  __shared__ __attribute__((aligned(256))) uint32_t s_ts[2][kGTsWords];

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  {  // token tiles per expert and their prefix (E <= 1024: 2 experts per thread)
    constexpr int PT = kMaxE / 512;
    int c[PT], tot = 0;
#pragma unroll
    for (int q = 0; q < PT; ++q) {
      const int e = tid * PT + q;
      c[q] = e < p.E && active(p, e) ? (p.offsets[e + 1] - p.offsets[e] + kGM - 1) / kGM : 0;
      tot += c[q];
    }
    int x = tot;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const int y = __shfl_up(x, off);
      if (lane >= off) x += y;
    }
    if (lane == 63) s_part[wave] = x;
    __syncthreads();
    int run = x - tot;
#pragma unroll
    for (int w = 0; w < 8; ++w)
      if (w < wave) run += s_part[w];
#pragma unroll
    for (int q = 0; q < PT; ++q) {
      const int e = tid * PT + q;
      if (e < p.E) s_pref[e] = run;
      run += c[q];
      if (e == p.E - 1) s_pref[p.E] = run;
    }
    __syncthreads();
  }
  const int total_items = s_pref[p.E] * n_ntiles;
  const int K = MODE == 0 ? p.d : p.f, R = MODE == 0 ? p.f : p.d;
  const int nk = (K + 127) >> 7, ss = mxfp8_scale_stride(K);
  const bool half = (K & 127) != 0;  // the last step holds 64 elements
  const size_t fd = (size_t)p.f * p.d;
  const int ng = gridDim.x, per_xcd = ng >> 3;
  const int pos = (blockIdx.x & 7) * per_xcd + (blockIdx.x >> 3);
  const int wn = wave & 3, wm = wave >> 2;
  const uint32_t lds_sm = g_lds_addr(sm), lds_ts = g_lds_addr(s_ts);
  const uint8_t* acodes = (const uint8_t*)(MODE == 0 ? p.x : p.h);

  for (int j = pos; j < total_items; j += ng) {
    const int q = j / n_ntiles;
    int lo = 0, hi = p.E;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (s_pref[mid] <= q) lo = mid; else hi = mid - 1;
    }
    const int e = lo;
    const int m_e = s_pref[e + 1] - s_pref[e];
    const int local = j - s_pref[e] * n_ntiles;
    const int grp = local / (4 * n_ntiles), first_m = grp * 4;
    const int gsz = min(4, m_e - first_m), in = local - grp * 4 * n_ntiles;
    const int nt = in / gsz, mt = first_m + (in - nt * gsz);
    const uint8_t* W = (const uint8_t*)entry_of(p, e);
    if (!W) continue;
    const int n0 = p.offsets[e] + mt * kGM;
    const int rows = min(kGM, p.offsets[e + 1] - n0);
    int ln = lane;
    asm volatile("" : "+v"(ln));  // keeps what follows from the lane out of the loops' live registers

    // A wave loads 32 token rows (four loads of 8 rows, a lane's 16-byte piece permuted), the codes
    // of two strips, the scales of four (waves w and w + 4 the same), and a load of a token scale
    // chunk: no branch, the same eight loads in each wave.  In a last step of 64 elements the second
    // half of a code tile and of its scales does not exist (the first is read twice); the pieces
    // of token rows past their end are other rows' or, at the buffer's last row, its last bytes.
    // None of that is used.
    auto row_at = [&](int r) {
      r = min(r, rows - 1);
      return (uint32_t)(MODE == 0 ? p.perm[n0 + r] / p.k : n0 + r);
    };
    uint32_t oa[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const int r = (4 * wave + t) * 8 + (ln >> 3);
      oa[t] = row_at(r) * (uint32_t)K + ((ln & 7) ^ ((r >> 1) & 7)) * 16;
    }
    const uint32_t ots = row_at(wave * 32 + (ln >> 2)) * (uint32_t)ss;
    const uint32_t ots_step = row_at(wave * 32 + 16 + (ln >> 2)) * (uint32_t)ss - ots;
    // first weight row of a group of four strips: 32 units of gate and of up, or 64 output channels
    // (past the matrix: the first ones, their results dropped)
    auto first_row = [&](int w) { return MODE == 0 ? nt * 128 + w * 32 : nt * 256 + w * 64; };
    const bool out = first_row(wn) < R;
    const int r0 = first_row(wn), rc = first_row(wave >> 1) < R ? first_row(wave >> 1) : 0, rs = out ? r0 : 0;
    const size_t strip = (size_t)K * 8;
    const uint8_t* const wcodes = W + (size_t)rc * (K / 2) + (MODE == 0 ? (wave & 1) * (fd / 2) : fd + (wave & 1) * 2 * strip);
    const uint8_t* const wscales = W + 3 * (fd / 2) + (MODE == 0 ? 0 : 2 * (fd / 32)) + (size_t)rs * (K / 32);
    const uint32_t ows = ((ln >> 4) & 1) * (K / 2) + (ln >> 5) * (uint32_t)(MODE == 0 ? fd / 32 : K) + (ln & 15) * 4;
    // Load i of 2 of the wave's part of token scale chunk c: rows 32 wave + 16 i .. + 15 (words past
    // a row's end: its last).
    auto issue_ts = [&](int c, int i) {
      const int n = min(c * 4 + ((ln & 3) ^ ((2 * wave + i) & 3)), (ss >> 2) - 1);
      g_load4(ascales, ots + i * ots_step + 4 * n, lds_ts + (c & 1) * (kGTsWords * 4) + (wave * 2 + i) * 256);
    };
    // The stage at LDS byte st <- step kt0 (at most nk - 1), and a load of the chunk that begins
    // two to five steps later (each of its loads is issued twice): the eight loads, two a quarter.
    auto issue = [&](uint32_t st, int kt0, auto quarter_tag) {
      constexpr int qt = decltype(quarter_tag)::value;
      const int kt = min(kt0, nk - 1);
      const bool sh = half && kt == nk - 1;
      if constexpr (qt < 2) {
#pragma unroll
        for (int t = 2 * qt; t < 2 * qt + 2; ++t)
          g_load16(acodes, min(oa[t] + (uint32_t)kt * 128, last_piece), st + kGTokAt + (4 * wave + t) * 1024);
      } else if constexpr (qt == 2) {
        const uint32_t oc = (sh ? ln & 31 : ln) * 16;
#pragma unroll
        for (int s = 0; s < 2; ++s)
          g_load16(wcodes + (size_t)kt * 1024 + s * strip, oc, st + kGCodeAt + (wave * 2 + s) * 1024);
      } else {
        g_load4(wscales + (size_t)kt * 64, ows - (sh ? (ln & 8) * 4 : 0), st + wn * 256);
        issue_ts((kt0 + 2) >> 2, kt0 & 1);
      }
    };
    using I0 = std::integral_constant<int, 0>;
    using I1 = std::integral_constant<int, 1>;
    using I2 = std::integral_constant<int, 2>;
    using I3 = std::integral_constant<int, 3>;

    // lane addresses of the operands (within a stage): token pieces by half step and piece, codes,
    // scales; token tile it of the wave is rows 64 it + 32 wm .. + 31
    const int g = ln >> 5, i32 = ln & 31;
    uint32_t at_tok[2][2];
#pragma unroll
    for (int kh = 0; kh < 2; ++kh)
#pragma unroll
      for (int c = 0; c < 2; ++c) at_tok[kh][c] = kGTokAt + (wm * 32 + i32) * 128 + ((4 * kh + 2 * c + g) ^ ((i32 >> 1) & 7)) * 16;
    const uint32_t at_code = kGCodeAt + wn * 4096 + (i32 >> 4) * 1024 + g * 256 + (i32 & 15) * 16;
    const uint32_t at_ws = wn * 256 + (i32 >> 4) * 64 + g * 16 + (i32 & 15);
    const uint32_t at_ts = lds_ts + (wm * 32 + i32) * 16, x_ts = ((2 * wm + (i32 >> 4)) & 3) * 4;

    f32x16 acc[2][4];
#pragma unroll
    for (int jn = 0; jn < 2; ++jn)
#pragma unroll
      for (int it = 0; it < 4; ++it)
#pragma unroll
        for (int v = 0; v < 16; ++v) acc[jn][it][v] = 0.f;

    // Operands: 64 elements of two token tiles, and of the wave's two weight tiles.
    struct Tokens {
      u32x4 t[2][2];
      uint32_t s[2];
    };
    struct Weights {
      u32x4 w[2];
      uint32_t s[2];
    };
    __syncthreads();  // the previous item's readers of the LDS are done
    issue_ts(0, 0);
    issue_ts(0, 1);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      issue(lds_sm + i * kGStage, i, I0{});
      issue(lds_sm + i * kGStage, i, I1{});
      issue(lds_sm + i * kGStage, i, I2{});
      issue(lds_sm + i * kGStage, i, I3{});
    }
    // AM token tiles in NP pairs; a step has NQ = 2 NP parts, part q = pair q % NP of half q / NP
    auto run_k = [&](auto am_tag) {
      constexpr int AM = decltype(am_tag)::value, NP = (AM + 1) / 2, NQ = 2 * NP;
      Tokens tk[2];
      Weights wt[2];
      auto read = [&](uint32_t st, int kt, auto q_tag) {
        constexpr int q = decltype(q_tag)::value, kh = q / NP, pr = q % NP;
        if (pr == 0) {
#pragma unroll
          for (int jn = 0; jn < 2; ++jn) {
            wt[kh].w[jn] = g_lds<u32x4>(at_code + st, jn * 2048 + kh * 512);
            wt[kh].s[jn] = g_lds<uint8_t>(at_ws + st, jn * 128 + kh * 32);
          }
        }
        // word of row r, step n of the chunk: n ^ (r / 16) mod 4, r = 64 it + 32 wm + i32
        const uint32_t ts = at_ts + ((kt >> 2) & 1) * (kGTsWords * 4) + (((kt & 3) * 4) ^ x_ts);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          if (2 * pr + u >= AM) continue;
          tk[q & 1].t[u][0] = g_lds<u32x4>(at_tok[kh][0] + st, (2 * pr + u) * 8192);
          tk[q & 1].t[u][1] = g_lds<u32x4>(at_tok[kh][1] + st, (2 * pr + u) * 8192);
          tk[q & 1].s[u] = g_lds<uint32_t>(ts, (2 * pr + u) * 1024);
        }
      };
      // The second half of a last step that has none: zeros (what was read may stand for NaN).
      auto blank = [&](auto q_tag) {
        constexpr int q = decltype(q_tag)::value, kh = q / NP, pr = q % NP;
        if (kh == 0) return;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          if (pr == 0) wt[kh].w[u] = half ? u32x4{0u, 0u, 0u, 0u} : wt[kh].w[u];
          if (pr == 0) wt[kh].s[u] = half ? 0u : wt[kh].s[u];
          if (2 * pr + u >= AM) continue;
          tk[q & 1].t[u][0] = half ? u32x4{0u, 0u, 0u, 0u} : tk[q & 1].t[u][0];
          tk[q & 1].t[u][1] = half ? u32x4{0u, 0u, 0u, 0u} : tk[q & 1].t[u][1];
          tk[q & 1].s[u] = half ? 0u : tk[q & 1].s[u];
        }
      };
      auto multiply = [&](auto q_tag) {
        constexpr int q = decltype(q_tag)::value, kh = q / NP, pr = q % NP;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          if (2 * pr + u >= AM) continue;
          const int ts = (int)(tk[q & 1].s[u] >> (8 * g));
#pragma unroll
          for (int jn = 0; jn < 2; ++jn)
            acc[jn][2 * pr + u] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                fp4_operand(wt[kh].w[jn]), fp8_operand(tk[q & 1].t[u][0], tk[q & 1].t[u][1]), acc[jn][2 * pr + u], 4, 0,
                0, (int)wt[kh].s[jn], 2 * kh, ts);
        }
      };
      using Q0 = std::integral_constant<int, 0>;
      using QL = std::integral_constant<int, NQ - 1>;
      // Part q's products over the reads of part q + 1, `loads` issued between.
      auto part = [&](uint32_t st, int kt, auto q_tag, auto loads) {
        constexpr int q = decltype(q_tag)::value;
        read(st, kt, std::integral_constant<int, (q + 1) % NQ>{});
        __builtin_amdgcn_sched_barrier(0);
        loads();
        multiply(q_tag);
        __builtin_amdgcn_sched_barrier(0);
      };
      using QL = std::integral_constant<int, NQ - 1>;
      using Q1 = std::integral_constant<int, 1 % NQ>;
      using Q2 = std::integral_constant<int, (NQ + 2) % NQ>;
      uint32_t st = lds_sm, st1 = lds_sm + kGStage, st2 = lds_sm + 2 * kGStage;
      issue(st2, 2, I0{});
      if constexpr (NQ == 2) issue(st2, 2, I1{});
      g_wait_loads<kGLoads + 8 / NQ>();
      lds_barrier();
      read(st, 0, Q0{});
      // A step: every part's operands are read under the products of the part before; ahead of
      // the last part's products the next step's stage is complete and this one's read by every
      // wave, and from there on to the same place of the next step the loads of the third step from
      // here go out (past the end: the last step's again, never read), some in each part: all at
      // once they hold a wave up until the address unit has taken them.
      for (int kt = 0; kt + 1 < nk; ++kt) {
        if constexpr (NQ == 4) {
          part(st, kt, Q0{}, [&] { issue(st2, kt + 2, I1{}); });
          part(st, kt, Q1{}, [&] { issue(st2, kt + 2, I2{}); });
          part(st, kt, Q2{}, [&] { issue(st2, kt + 2, I3{}); });
        } else {
          part(st, kt, Q0{}, [&] {
            issue(st2, kt + 2, I2{});
            issue(st2, kt + 2, I3{});
          });
        }
        g_wait_loads<kGLoads>();
        lds_barrier();
        part(st1, kt + 1, QL{}, [&] {
          issue(st, kt + 3, I0{});
          if constexpr (NQ == 2) issue(st, kt + 3, I1{});
        });
        const uint32_t t = st;
        st = st1;
        st1 = st2;
        st2 = t;
      }
      auto none = [] {};
      part(st, nk - 1, Q0{}, none);
      blank(Q1{});
      if constexpr (NQ == 4) {
        part(st, nk - 1, Q1{}, none);
        blank(Q2{});
        part(st, nk - 1, Q2{}, none);
        blank(QL{});
      }
      multiply(QL{});
      g_wait_loads<0>();  // those past the end too: the next item's may not be overtaken
    };
    switch ((rows + 63) >> 6) {
      case 1: run_k(std::integral_constant<int, 1>{}); break;
      case 2: run_k(std::integral_constant<int, 2>{}); break;
      case 3: run_k(std::integral_constant<int, 3>{}); break;
      default: run_k(std::integral_constant<int, 4>{}); break;
    }

    // lane 32 g + i, value v: token row i, weight row 8 (v / 4) + 4 g + v % 4 of the tile's 32
#pragma unroll
    for (int it = 0; it < 4; ++it) {
      if (it * 64 + wm * 32 >= rows || !out) continue;
      const int r = it * 64 + wm * 32 + i32;
      if (MODE == 0) {
        const int u0 = r0;
        float h[16];
        uint32_t m = 0;
#pragma unroll
        for (int v = 0; v < 16; ++v) {
          h[v] = g_swiglu(acc[0][it][v], acc[1][it][v]);
          m = max(m, abs_bits(h[v]));
        }
        m = max(m, (uint32_t)__shfl_xor((int)m, 32));
        const uint32_t s = mxfp8_scale_of(m);
        const float sc = e8m0_value(s);
        uint32_t w[4];
#pragma unroll
        for (int b = 0; b < 4; ++b) w[b] = mxfp8_pack4(h[4 * b], h[4 * b + 1], h[4 * b + 2], h[4 * b + 3], s, sc);
        g_pair_rows(w);
        if (r < rows) {
          *(u32x4*)((uint8_t*)p.h + (size_t)(n0 + r) * p.f + u0 + 16 * g) = u32x4{w[0], w[1], w[2], w[3]};
          if (g == 0) hscales[(size_t)(n0 + r) * mxfp8_scale_stride(p.f) + (u0 >> 5)] = (uint8_t)s;
        }
      } else {
#pragma unroll
        for (int jn = 0; jn < 2; ++jn) {
          const int o0 = r0 + jn * 32;
          const size_t at = (size_t)(n0 + r) * p.d + o0;
          if (YDT == MOE_F32) {
            if (r < rows) {
#pragma unroll
              for (int b = 0; b < 4; ++b)
                *(f32x4*)((float*)p.y + at + 8 * b + 4 * g) = f32x4{acc[jn][it][4 * b], acc[jn][it][4 * b + 1],
                                                                    acc[jn][it][4 * b + 2], acc[jn][it][4 * b + 3]};
            }
          } else {
            uint32_t a[4], c[4];  // elements 8 b + 4 g .. + 1 and + 2 .. + 3
#pragma unroll
            for (int b = 0; b < 4; ++b) {
              a[b] = (uint32_t)f32_to_bf16(acc[jn][it][4 * b]) | (uint32_t)f32_to_bf16(acc[jn][it][4 * b + 1]) << 16;
              c[b] = (uint32_t)f32_to_bf16(acc[jn][it][4 * b + 2]) | (uint32_t)f32_to_bf16(acc[jn][it][4 * b + 3]) << 16;
            }
            g_pair_rows(a);
            g_pair_rows(c);
            if (r < rows) {
              uint16_t* y = (uint16_t*)p.y + at + 16 * g;
              *(u32x4*)y = u32x4{a[0], c[0], a[1], c[1]};
              *(u32x4*)(y + 8) = u32x4{a[2], c[2], a[3], c[3]};
            }
          }
        }
      }
    }
  }
}

}  // namespace

// Token rows and h rows are addressed with 32-bit byte offsets.
bool ffn_mx8_gemm_supported(long long T, int k, int d, int f) {
  return T * d <= (1ll << 32) && T * k * f <= (1ll << 32);
}

int launch_ffn_mx8_gemm(const FfnArgs& p, int T, int y_dtype, hipStream_t stream) {
  const uint8_t* xs = (const uint8_t*)p.x + (size_t)T * p.d;
  uint8_t* hs = (uint8_t*)p.h + (size_t)T * p.k * p.f;
  const dim3 grid((num_cus() + 7) / 8 * 8), blk(512);
  const int ntd = (p.d + 255) / 256;
  const uint32_t last_h = (uint32_t)((size_t)T * p.k * p.f - 16);
  hipLaunchKernelGGL((m8_tile<0, MOE_BF16>), grid, blk, 0, stream, p, xs, (uint32_t)((size_t)T * p.d - 16), hs, (p.f + 127) / 128);
  MOE_LAUNCH_CHECK();
  if (y_dtype == MOE_F32) hipLaunchKernelGGL((m8_tile<1, MOE_F32>), grid, blk, 0, stream, p, hs, last_h, nullptr, ntd);
  else hipLaunchKernelGGL((m8_tile<1, MOE_BF16>), grid, blk, 0, stream, p, hs, last_h, nullptr, ntd);
  MOE_LAUNCH_CHECK();
  return MOE_OK;
}

}  // namespace moe
