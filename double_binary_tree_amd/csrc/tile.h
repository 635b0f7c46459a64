// Matrix tiles on the matrix cores: C[m][n] = sum_k A[m][k] * B[n][k] for one
// workgroup's BM x BN tile, both operands k-contiguous, sums in f32.
//
// Staging.  One k-step covers 128 bytes of every row (64 16-bit or 32 f32
// values).  Rows go from global memory straight to LDS, 16 bytes a lane, one
// 1 KiB wave access holding 8 rows; two stages alternate, so the loads of
// step s + 1 run while step s is multiplied.  The 16-byte chunk c of row r
// sits at chunk c ^ ((r >> 1) & 7): the 16 rows that a matrix instruction
// reads at one chunk then cover all 64 banks once (a row spans 32 banks, so
// rows r and r + 1 differ in the half, rows r and r + 2 in the chunk).  The
// permutation is applied to the global address, since LDS is filled in lane
// order.
//
// Ragged edges.  Rows past the operand's last one read the last row again
// (their results are dropped by the caller).  A k extent is a whole number
// of 16-byte chunks; in a last step that is not whole the missing chunks are
// loaded from the row's last chunk and overwritten by zeros in LDS.
#pragma once

#include "device_ops.h"

namespace emu {

constexpr int kStepBytes = 128;   // bytes of k per stage and row

// What a matrix instruction multiplies: 16 bytes of a row per lane.
template <DType T>
struct Mma;
template <>
struct Mma<DType::F16> {
  static __device__ __forceinline__ void mul(u32x4 a, u32x4 b, f32x4& c) {
    c = __builtin_amdgcn_mfma_f32_16x16x32_f16(bits<f16x8>(a), bits<f16x8>(b), c, 0, 0, 0);
  }
};
template <>
struct Mma<DType::BF16> {
  static __device__ __forceinline__ void mul(u32x4 a, u32x4 b, f32x4& c) {
    c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bits<bf16x8>(a), bits<bf16x8>(b), c, 0, 0, 0);
  }
};
// Four k values a lane: value i of the lanes of group g (lane >> 4) is k =
// 4g + i in both operands, so instruction i sums k = i, 4 + i, 8 + i, 12 + i.
template <>
struct Mma<DType::F32> {
  static __device__ __forceinline__ void mul(u32x4 a, u32x4 b, f32x4& c) {
    const f32x4 x = bits<f32x4>(a), y = bits<f32x4>(b);
#pragma unroll
    for (int i = 0; i < 4; ++i) c = __builtin_amdgcn_mfma_f32_16x16x4f32(x[i], y[i], c, 0, 0, 0);
  }
};

// One operand of a tile: `base` is the tile's first row at k = 0 (uniform),
// `ld` the row pitch in bytes, `rows` how many rows are left (>= 1).
struct Operand {
  const char* base;
  uint32_t ld;
  int rows;
};

// 16 bytes per lane from base + off to LDS at `lds` + 16 * lane (base and lds
// uniform).  Written as assembly because the compiler takes every LDS read
// after the builtin as possibly reading what the load writes and waits for
// all loads first, which would undo the double buffering; the load has no
// register output, and lds_arrived() is the wait that goes with it.
__device__ __forceinline__ void load_to_lds(const char* base, uint32_t off, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(lds), "v"(off), "s"(base)
               : "memory");
}
// This wave's loads to LDS have all arrived (other waves': after a barrier).
__device__ __forceinline__ void lds_arrived() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }
// LDS by byte address (an address-space cast of a generic pointer per access
// would leave the compiler with flat accesses).
typedef __attribute__((address_space(3))) u32x4 LdsVec;
__device__ __forceinline__ uint32_t lds_address(const void* p) {
  return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) char*)p;
}
__device__ __forceinline__ u32x4 lds_read(uint32_t at) { return *(const LdsVec*)(uintptr_t)at; }
__device__ __forceinline__ void lds_write(uint32_t at, u32x4 v) { *(LdsVec*)(uintptr_t)at = v; }

// BM x BN by WGM x WGN waves, each wave MF x NF fragments of 16 x 16.
// acc[i][j] of a lane holds C[m][n] at m = 16 i + 4 (lane >> 4) + e, n = 16 j
// + (lane & 15) of the wave's part, e = 0 .. 3.
template <DType T, int BM_, int BN_, int WGM_, int WGN_>
struct TileMma {
  static constexpr int BM = BM_, BN = BN_, WGM = WGM_, WGN = WGN_;
  static constexpr int waves = WGM * WGN, threads = 64 * waves;
  static constexpr int WM = BM / WGM, WN = BN / WGN, MF = WM / 16, NF = WN / 16;
  static constexpr int stage_bytes = (BM + BN) * kStepBytes;
  static constexpr int lds_bytes = 2 * stage_bytes;
  static constexpr int LA = BM / 8 / waves, LB = BN / 8 / waves;   // loads per wave and stage
  static_assert(LA * 8 * waves == BM && LB * 8 * waves == BN, "whole wave accesses");
  using Acc = f32x4[MF][NF];

  // Byte offset of this lane's chunk of load l (0 .. n-1 of the wave) from
  // the operand's base at k = 0, and whether the chunk lies in `chunks`.
  template <int L>
  static __device__ __forceinline__ void offsets(const Operand& o, int wave, int lane, int chunks, uint32_t (&off)[L],
                                                 bool (&pad)[L]) {
#pragma unroll
    for (int l = 0; l < L; ++l) {
      const int r = (wave * L + l) * 8 + (lane >> 3);
      const int c = (lane & 7) ^ ((r >> 1) & 7);
      pad[l] = c >= chunks;
      off[l] = (uint32_t)min(r, o.rows - 1) * o.ld + 16u * (uint32_t)min(c, chunks - 1);
    }
  }

  static __device__ __forceinline__ void stage(const Operand& a, const Operand& b, const uint32_t (&oa)[LA],
                                               const uint32_t (&ob)[LB], uint64_t k, uint32_t lds, int wave) {
#pragma unroll
    for (int l = 0; l < LA; ++l) load_to_lds(a.base + k, oa[l], lds + (wave * LA + l) * 1024);
#pragma unroll
    for (int l = 0; l < LB; ++l) load_to_lds(b.base + k, ob[l], lds + BM * kStepBytes + (wave * LB + l) * 1024);
  }

  static __device__ __forceinline__ void multiply(uint32_t lds, int wm, int wn, int lane, Acc& acc) {
    const int r = lane & 15, g = lane >> 4;
    const uint32_t pa = lds + (wm * WM + r) * kStepBytes;
    const uint32_t pb = lds + BM * kStepBytes + (wn * WN + r) * kStepBytes;
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
      const int c = ((kk * 4 + g) ^ ((r >> 1) & 7)) * 16;
      u32x4 fa[MF], fb[NF];
#pragma unroll
      for (int j = 0; j < NF; ++j) fb[j] = lds_read(pb + j * 16 * kStepBytes + c);
#pragma unroll
      for (int i = 0; i < MF; ++i) fa[i] = lds_read(pa + i * 16 * kStepBytes + c);
#pragma unroll
      for (int i = 0; i < MF; ++i)
#pragma unroll
        for (int j = 0; j < NF; ++j) Mma<T>::mul(fa[i], fb[j], acc[i][j]);
    }
  }

  // Adds A * B^T over `kbytes` bytes of k (a multiple of 16, > 0) to acc.
  // On return every wave may still be reading `lds`.
  static __device__ __forceinline__ void run(const Operand& a, const Operand& b, uint64_t kbytes, uint32_t lds, Acc& acc) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / WGN, wn = wave % WGN;
    const uint32_t steps = (uint32_t)((kbytes + kStepBytes - 1) / kStepBytes);
    const int last = (int)((kbytes - (uint64_t)(steps - 1) * kStepBytes) / 16);   // chunks of the last step
    uint32_t oa[LA], ob[LB], ta[LA], tb[LB];
    bool pa[LA], pb[LB];
    offsets<LA>(a, wave, lane, 8, oa, pa);
    offsets<LB>(b, wave, lane, 8, ob, pb);
    offsets<LA>(a, wave, lane, last, ta, pa);
    offsets<LB>(b, wave, lane, last, tb, pb);
    auto fetch = [&](uint32_t s) {
      const uint32_t to = lds + (s & 1) * stage_bytes;
      if (s + 1 < steps || last == 8) stage(a, b, oa, ob, (uint64_t)s * kStepBytes, to, wave);
      else stage(a, b, ta, tb, (uint64_t)s * kStepBytes, to, wave);
    };
    fetch(0);
    for (uint32_t s = 0; s < steps; ++s) {
      lds_arrived();
      __syncthreads();     // step s is in LDS; every wave is done with the other stage
      const uint32_t at = lds + (s & 1) * stage_bytes;
      if (s + 1 < steps) {
        fetch(s + 1);
      } else if (last != 8) {
        const u32x4 zero = {0, 0, 0, 0};
#pragma unroll
        for (int l = 0; l < LA; ++l)
          if (pa[l]) lds_write(at + (wave * LA + l) * 1024 + lane * 16, zero);
#pragma unroll
        for (int l = 0; l < LB; ++l)
          if (pb[l]) lds_write(at + BM * kStepBytes + (wave * LB + l) * 1024 + lane * 16, zero);
        __syncthreads();
      }
      multiply(at, wm, wn, lane, acc);
    }
  }
};

// Workgroup -> tile.  Consecutive workgroups go to the 8 XCDs in turn, so
// workgroup w of `total` is taken as the (w / 8)-th of XCD w % 8's contiguous
// share, and the tiles are walked in bands of `band` tile rows: the tiles
// that one XCD works on at a time share rows of both operands in its L2.
__device__ __forceinline__ void tile_of(uint32_t w, uint32_t tm, uint32_t tn, uint32_t band, uint32_t& m, uint32_t& n) {
  const uint32_t total = tm * tn, x = w & 7, q = total >> 3, rem = total & 7;
  uint32_t t = x * q + min(x, rem) + (w >> 3);
  const uint32_t per = band * tn, g = t / per, first = g * band, rows = min(band, tm - first);
  t -= g * per;
  m = first + t % rows;
  n = t / rows;
}

}  // namespace emu
