// gemm_linear_epilogue.hpp -- the linear layer's epilogue on a wave's
// accumulator tile (included by gemm_linear.hpp):
//   z = alpha * scale_a[m] * scale_b[n] * acc + bias[n]
//   Z = z (if kept),  D = act(z) + R
// (LIN 2: D = alpha * acc + R)
// in fp32 on the unrounded accumulator (int32 sums are converted first),
// rounded to nearest-even into the type T that D, R and Z share.
//
// Same re-layout through LDS as the one-type epilogue: a lane keeps the same
// VEC columns through all passes, so bias[n] and alpha * scale_b[n] are read
// once per tile into registers; residual and row scales are loaded four or
// eight passes ahead of their use.  With activations the passes of a large
// tile's block run in a loop of four: the five expanded in every pass would
// take several times the 64 KiB instruction cache.  (A loop over the blocks as well makes
// the accumulators loop-carried, and they spill.)
#pragma once

namespace gemm_epi {

template <class CF, int T, class ACC>
__device__ __forceinline__ void epilogue_linear(const LinParams& p, const ACC (&acc)[CF::FM][CF::FN], char* lds,
                                                int wave, int lane, int mw, int nw) {
  constexpr int LINE = CF::epi_line(true), PITCH = CF::epi_pitch(true);
  constexpr int ES = EpiElem<T>::SIZE;
  constexpr int VEC = 16 / ES;
  constexpr int LPL = LINE / VEC;
  constexpr int LPP = 64 / LPL;  // lines (rows) per pass
  static_assert(LPL >= 1 && LPL <= 64 && 32 % LPP == 0, "line split over the lanes");
  constexpr int NBLK = CF::WM / 32;
  constexpr int PASSES = 32 / LPP;
  float* region = (float*)(lds + wave * CF::epi_wave_bytes(true));
  const int sub = lane / LPL;
  const int e = (lane % LPL) * VEC;

  const int64_t lines = min(max(p.M - mw, (int64_t)0), (int64_t)CF::WM);
  const int along = nw + e;
  const bool lane_ok = along < p.N;
  // rows past the matrix lie outside a resource's extent, lanes past its
  // columns get an offset above 2^31; a tensor that is not there has an empty
  // resource
  auto rsrc = [&](const void* base, int64_t ld) {
    return __builtin_amdgcn_make_buffer_rsrc(base ? (void*)((const char*)base + mw * ld * ES) : (void*)p.D, (short)0,
                                             base ? (int)(lines * ld * ES) : 0, 0x00020000);
  };
  const __amdgpu_buffer_rsrc_t rd = rsrc(p.D, p.ldd), rr = rsrc(p.R, p.ldr), rz = rsrc(p.Z, p.ldz);
  auto lane_off = [&](int64_t ld) { return lane_ok ? (uint32_t)((sub * ld + along) * ES) : 0x80000000u; };
  const uint32_t od = lane_off(p.ldd), orr = lane_off(p.ldr), oz = lane_off(p.ldz);
  const uint32_t sd = (uint32_t)(LPP * p.ldd * ES), sr = (uint32_t)(LPP * p.ldr * ES), sz = (uint32_t)(LPP * p.ldz * ES);
  const __amdgpu_buffer_rsrc_t rsa = __builtin_amdgcn_make_buffer_rsrc(
      p.scale_a ? (void*)(p.scale_a + mw) : (void*)p.D, (short)0, p.scale_a ? (int)(lines * 4) : 0, 0x00020000);

  // The passes of a block run in a loop of UN, or unrolled where that stays
  // small; residual and row scales run AHEAD passes ahead.
  constexpr int NP = NBLK * PASSES;
  constexpr int UN = CF::LIN_ACT && NBLK > 2 ? 4 : PASSES < 8 ? PASSES : 8;
  constexpr int AHEAD = PASSES == UN ? (NP < 8 ? NP : 8) : UN;
  static_assert(PASSES % UN == 0, "passes in groups");
  v4u res[AHEAD];
  float sa[AHEAD];
  auto fetch = [&](int pass, auto u_c) {
    constexpr int u = decltype(u_c)::value;
    if (p.R) res[u] = epi_ld<T>(rr, orr + (uint32_t)pass * sr);
    if (CF::LIN_ACT && p.scale_a)
      sa[u] = __uint_as_float((uint32_t)__builtin_amdgcn_raw_buffer_load_b32(rsa, (pass * LPP + sub) * 4, 0, 0));
  };
  static_for<0, AHEAD>([&](auto u_c) {
    res[decltype(u_c)::value] = v4u{};
    sa[decltype(u_c)::value] = 1.0f;
    fetch(decltype(u_c)::value, u_c);
  });

  // this lane's columns
  float bias[VEC], cs[VEC];
#pragma unroll
  for (int i = 0; i < VEC; ++i) bias[i] = 0.0f, cs[i] = p.alpha;
  if (CF::LIN_ACT && lane_ok) {
    if (p.scale_b) {
#pragma unroll
      for (int i = 0; i < VEC; ++i) cs[i] = p.alpha * p.scale_b[along + i];
    }
    if (p.bias) {
      if (p.bias_dtype == T_F32) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) bias[i] = ((const float*)p.bias)[along + i];
      } else if (p.bias_dtype == T_F16) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) bias[i] = (float)((const _Float16*)p.bias)[along + i];
      } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) bias[i] = (float)((const __bf16*)p.bias)[along + i];
      }
    }
  }

  static_for<0, NBLK>([&](auto blk_c) {
    constexpr int blk = decltype(blk_c)::value;
    // this wave's reads of the previous block are issued before these writes,
    // and LDS serves one wave's operations in order
    epi_stage_block<CF, true>(acc, region, lane, blk);
#pragma unroll 1
    for (int g = 0; g < PASSES; g += UN) static_for<0, UN>([&](auto u_c) {
      constexpr int u = decltype(u_c)::value;
      const int pass = blk * PASSES + g + u;
      const float* wp = region + ((g + u) * LPP + sub) * PITCH + e;
      float v[VEC];
#pragma unroll
      for (int i = 0; i < VEC; i += 4) {
        const v4f w = *(const v4f*)(wp + i);
#pragma unroll
        for (int j = 0; j < 4; ++j) v[i + j] = CF::INT ? (float)__float_as_int(w[j]) : w[j];
      }
      constexpr int slot = PASSES == UN ? (blk * PASSES + u) % AHEAD : u;
      const v4u r = res[slot];
      const float s = sa[slot];
      if (pass + AHEAD < NP) fetch(pass + AHEAD, IntC<slot>{});
#pragma unroll
      for (int i = 0; CF::LIN_ACT && i < VEC; ++i) v[i] = __builtin_fmaf(v[i], s * cs[i], bias[i]);
      auto pack = [&](const float (&x)[VEC]) {
        return epi_pack<T>(v4f{x[0], x[1], x[2], x[3]},
                           VEC == 8 ? v4f{x[VEC - 4], x[VEC - 3], x[VEC - 2], x[VEC - 1]} : v4f{});
      };
      if (CF::LIN_ACT && p.Z) epi_st<T>(rz, oz + (uint32_t)pass * sz, pack(v));
      if constexpr (CF::LIN_ACT) with_act(p.act, [&](auto act_c) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) v[i] = act_value<decltype(act_c)::value>(v[i]);
      });
      // (a branch: multiplying by 1 adds 0.9 us to the backward of 4096^3, 235.5)
      if (!CF::LIN_ACT && p.alpha != 1.0f) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) v[i] *= p.alpha;
      }
      if (p.R) {
#pragma unroll
        for (int i = 0; i < VEC; i += 4) {
          const v4f d = epi_dec<T>(r, i / 4);
#pragma unroll
          for (int j = 0; j < 4; ++j) v[i + j] += d[j];
        }
      }
      epi_st<T>(rd, od + (uint32_t)pass * sd, pack(v));
      __builtin_amdgcn_sched_barrier(0);  // passes stay in program order
    });
  });
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
}

}  // namespace gemm_epi
