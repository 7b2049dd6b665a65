// Weight gradient from an 8-bit checkpoint on gfx950 matrix cores:
//
//   grad_w[n][k] = sum over rows m of gy[m][n] * x[m][k],   x = E4M3 code * 2^(s - 127)
//
// gy is bf16 as it arrives; a code times its power of two is exact in bf16, so the bf16
// MFMA multiplies the checkpoint's values exactly and accumulates in fp32: nothing is
// rounded before the sum.
//
// Both operands have the contraction (rows) as their slow dimension, while an MFMA lane
// needs consecutive contraction values of one column.  The transposition costs nothing:
// LDS holds the tiles as they are in memory, [64 rows][256 columns] of bf16, and
// ds_read_b64_tr_b16 hands each lane four rows of its column.
//
// A 256-thread workgroup owns a square tile of grad_w, each of its four waves a quarter in
// kT x kT tiles of v_mfma_f32_32x32x16_bf16: kT = 4 gives 256 x 256 (one wave per SIMD),
// kT = 2 gives 128 x 128 (two workgroups per compute unit) for products with too few large
// tiles.  Rows advance in steps of 64 through two LDS stages:
//   * gy goes global -> LDS directly, 16 bytes a lane, where its rows are aligned to that;
//     else through registers in 16-byte loads at any address (777 rows, 1023 x 5120: 23.8 us,
//     in 2-byte loads 63; 4096 rows, 5121 x 5120: 242 and 1128; 5120 x 5120 aligned: 203);
//   * codes go through registers: loaded a step ahead, expanded by the hardware's scaled
//     conversion (one instruction per two values), written to LDS as bf16;
//   * copies and code loads are buffer loads, whose range check supplies zeros for rows and
//     columns past the end: they add nothing even where gy holds infinities, and the loop
//     carries no per-lane address arithmetic;
//   * a row of a panel is chunks of 16 bytes, chunk c at position c ^ 4 (row % 4) (the
//     four rows that one transposed read gathers lie in different banks), for x with bit 0
//     also flipped by bit 3 of c (so that the 32-byte writes of neighbouring lanes do).
// Few tiles (a narrow projection) leave compute units idle, so the rows are split across
// workgroups into fp32 partials that weight_grad_reduce adds in split order.
//
// Measured, 4096 rows, 25600 x 5120: 900-990 us, 1.09-1.19 PFLOP/s, by the box.  The matrix
// cores are busy 57 % of the cycles, at a clock that falls from 1.9 to 1.5 GHz over calls
// in a row.  The same launch on zeros takes 766 us, 100 of them the 524 MB that the epilogue
// writes while every compute unit is at the same place, 115 the codes and 50 the copies of
// gy.  777 rows, 1024 x 5120 in small tiles: 18-21 us, 13.5 of them without any operand
// loads (launch, 21 MB of output, and LDS reads that match the MFMAs' rate).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "checkpoint_device.h"
#include "gemm_common.h"
#include "nvfp4_device.h"
#include "nvfp4_launch.h"

namespace nvfp4 {
namespace {

typedef float float16_t __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef short short4_t __attribute__((ext_vector_type(4)));
typedef short short8_t __attribute__((ext_vector_type(8)));

constexpr int kStep = 64;                   // rows per LDS stage
template <int kT>
struct Geo {
  static constexpr int kTile = 64 * kT;                // columns of gy, and of x, per workgroup
  static constexpr int kRowBytes = kTile * 2;
  static constexpr int kPanel = kStep * kRowBytes;     // one operand of one stage
  static constexpr int kLds = 4 * kPanel;              // 128 KB or 64 KB
  static constexpr int kRowChunks = kTile / 8;         // 16-byte chunks of a panel row
  static constexpr int kCopyRows = 64 / kRowChunks;    // rows one copy instruction of a wave fills
  static constexpr int kXChunks = kTile / 16;          // 16-code chunks of a row
  static constexpr int kXRows = 256 / kXChunks;        // rows of codes the workgroup loads at a time
  static constexpr int kOutRow = 32 * kT + 4;          // words per staged output row
  static_assert(kStep / kXRows == kT && kStep / (4 * kCopyRows) == 2 * kT, "passes");
  static_assert(4 * 32 * kOutRow * 4 <= kLds, "output staging fits");
};
constexpr int kBand = 4;                    // tile rows per band of the tile order

// Position of chunk c in row r.
__device__ __forceinline__ int swz(int r, int c) { return c ^ ((r & 3) << 2); }
__device__ __forceinline__ int swz_x(int r, int c) { return swz(r, c) ^ ((c >> 3) & 1); }

// A buffer of `bytes` bytes from p (wave-uniform): loads past them return zero.
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
__device__ __forceinline__ u32x4_t buffer_of(const void* p, uint32_t bytes) {
  const uint64_t a = (uint64_t)p;
  return u32x4_t{(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)a),
                 (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(a >> 32) & 0xFFFF),
                 (uint32_t)__builtin_amdgcn_readfirstlane((int)bytes), 0x00020000u};
}
constexpr uint32_t kOutside = 0x80000000u;   // an offset past every buffer here
constexpr int64_t kBufferWidth = 1 << 24;    // columns up to which a step's rows fit 31-bit offsets

// One 16-byte global -> LDS copy per lane; the address is a wave-uniform LDS base plus
// 16 bytes a lane.  Inline asm so that the compiler does not hold LDS reads back for it: the
// loop waits for it before the barrier that precedes them.
__device__ __forceinline__ void copy16_to_lds(u32x4_t rsrc, uint32_t offset, uint8_t* dst) {
  asm volatile("buffer_load_dwordx4 %1, %2, 0 offen lds"
               :: "{m0}"((uint32_t)(uintptr_t)dst), "v"(offset), "s"(rsrc) : "memory");
}
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc_of(const void* p, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, (int)bytes, 0x00020000);
}
__device__ __forceinline__ void step_barrier() {
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// A barrier for panels whose copies each wave has waited for already.
__device__ __forceinline__ void panel_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// Scheduling of a group of MFMAs: kN times an MFMA, kReads LDS reads and some vector work.
template <int kN, int kReads>
__device__ __forceinline__ void interleave() {
#pragma unroll
  for (int g = 0; g < kN; ++g) {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    __builtin_amdgcn_sched_group_barrier(0x100, kReads, 0);
    __builtin_amdgcn_sched_group_barrier(0x002, 3, 0);
  }
  __builtin_amdgcn_sched_barrier(0);
}

// Four rows of one column (see the lane layout at the reads below).
__device__ __forceinline__ short4_t read_tr(const uint8_t* p) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) short4_t*)p);
}

// 16 codes -> 32 bytes of bf16.
__device__ __forceinline__ void expand16(const u32x4_t& w, float scale, uint4 (&o)[2]) {
  uint32_t r[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    r[2 * i] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[i], scale, false));
    r[2 * i + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[i], scale, true));
  }
  o[0] = make_uint4(r[0], r[1], r[2], r[3]);
  o[1] = make_uint4(r[4], r[5], r[6], r[7]);
}

// How gy comes:
//   kCopy    its rows start on 16-byte boundaries (N a multiple of 8): copied to LDS;
//   kLoad    at least 8 columns: through registers, in 16-byte loads of any alignment;
//   kGather  value by value: narrower still, no rows, or an N or K whose rows of a step do
//            not fit the 31-bit offsets of the others.
enum Gy { kCopy, kLoad, kGather };
template <int kT, Gy kGy, bool kOutBf16>
__global__ void __launch_bounds__(256, kT == 4 ? 1 : 2) weight_grad_kernel(
    const uint16_t* __restrict__ gy, int64_t m, int64_t n, const uint8_t* __restrict__ codes,
    const uint8_t* __restrict__ scales, int64_t k, void* __restrict__ out, int tiles_n, int tiles_k, int splits,
    float* __restrict__ partial) {
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  using G = Geo<kT>;
  constexpr int kTile = G::kTile, kRowBytes = G::kRowBytes, kPanel = G::kPanel;
  // Workgroups are dealt round-robin to the 8 XCDs: each XCD gets a contiguous run of
  // tiles, ordered in bands of kBand tile rows, so the tiles resident on one XCD share
  // operand columns in its L2.  With splits, the splits of a tile follow each other.
  const int nblk = gridDim.x;
  int bid = blockIdx.x;
  if ((nblk & 7) == 0) bid = (bid & 7) * (nblk >> 3) + (bid >> 3);
  const int split = bid % splits;
  bid /= splits;
  const int band = bid / (kBand * tiles_k);
  const int band_rows = min(tiles_n - band * kBand, kBand);
  const int in_band = bid - band * kBand * tiles_k;
  const int64_t n0 = (int64_t)(band * kBand + in_band % band_rows) * kTile;
  const int64_t k0 = (int64_t)(in_band / band_rows) * kTile;

  const int t = threadIdx.x;
  const int lane = t & 63;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int wn = wave >> 1, wk = wave & 1;
  const int64_t steps = (m + kStep - 1) / kStep;
  const int64_t s_begin = steps * split / splits, s_end = steps * (split + 1) / splits;
  const int64_t kb = (k + kCkBlock - 1) / kCkBlock;

  auto panel_a = [&](int64_t s) { return lds + (int)(s & 1) * 2 * kPanel; };
  auto panel_b = [&](int64_t s) { return lds + (int)(s & 1) * 2 * kPanel + kPanel; };

  // bytes of the rows of step s in an array of `width` bytes a row
  auto step_bytes = [&](int64_t s, int64_t width) {
    const int64_t rows = s < s_end ? min(m - s * kStep, (int64_t)kStep) : 0;
    return (uint32_t)(rows * width);
  };
  // gy, kCopy: instruction i of wave w fills rows (2 kT w + i) kCopyRows .. of the panel; the
  // others: chunk 256 i + t of the panel.
  uint32_t goff[2 * kT];
#pragma unroll
  for (int i = 0; i < 2 * kT; ++i) {
    if constexpr (kGy == kCopy) {
      const int r = (2 * kT * wave + i) * G::kCopyRows + lane / G::kRowChunks;
      const int64_t col = n0 + 8 * swz(r, lane % G::kRowChunks);
      goff[i] = col < n ? (uint32_t)((r * n + col) * 2) : kOutside;
    } else {
      const int r = (256 * i + t) / G::kRowChunks;
      goff[i] = (uint32_t)((r * n + min(n0 + 8 * (t % G::kRowChunks), n - 1)) * 2);
    }
  }
  auto stage_gy = [&](int64_t s, int i) {
    uint8_t* dst = panel_a(s);
    if constexpr (kGy == kCopy) {
      copy16_to_lds(buffer_of(gy + s * kStep * n, step_bytes(s, 2 * n)), goff[i], dst + (2 * kT * wave + i) * 1024);
    } else {
      const int r = (256 * i + t) / G::kRowChunks, c = t % G::kRowChunks;
      const int64_t row = s * kStep + r;
      uint32_t w[4] = {0, 0, 0, 0};
      if (s < s_end && row < m) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int64_t col = n0 + 8 * c + e;
          if (col < n) w[e >> 1] |= (uint32_t)gy[row * n + col] << (16 * (e & 1));
        }
      }
      *reinterpret_cast<uint4*>(dst + r * kRowBytes + swz(r, c) * 16) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  };
  // kLoad: what follows a row in memory comes along in its last chunk, and chunks past it
  // repeat it: both meet only columns past the last, which are not written.  Loads that would
  // pass the tensor's end move back to it; trim_gy shifts what they hold into place and
  // clears rows past the last.
  u32x4_t gr[kGy == kLoad ? 2 * kT : 1];
  auto bytes_left = [&](int64_t s) { return (uint32_t)min((m - s * kStep) * n * 2, (int64_t)0x7FFFFFFF); };
  auto load_gy = [&](int64_t s, int i) {
    s = min(s, steps - 1);   // past the last step: loaded, not used
    __builtin_memcpy(&gr[i], reinterpret_cast<const uint8_t*>(gy + s * kStep * n) + min(goff[i], bytes_left(s) - 16), 16);
  };
  auto trim_gy = [&](int64_t s) {
    const uint32_t left = bytes_left(min(s, steps - 1));
    if (left >= (uint32_t)kStep * 2 * (uint32_t)n + 16) return;
#pragma unroll
    for (int i = 0; i < 2 * kT; ++i) {
      const uint32_t d = goff[i] - min(goff[i], left - 16);   // bytes moved back
      const uint64_t lo = gr[i][0] | (uint64_t)gr[i][1] << 32, hi = gr[i][2] | (uint64_t)gr[i][3] << 32;
      const uint32_t sh = 8 * (d & 7);
      const uint64_t hs = hi >> sh, ls = sh ? (lo >> sh) | (hi << (64 - sh)) : lo;
      const uint64_t a = d < 8 ? ls : d < 16 ? hs : 0, b = d < 8 ? hs : 0;
      gr[i] = u32x4_t{(uint32_t)a, (uint32_t)(a >> 32), (uint32_t)b, (uint32_t)(b >> 32)};
    }
  };
  auto store_gy = [&](int64_t s, int i) {
    const int r = (256 * i + t) / G::kRowChunks, c = t % G::kRowChunks;
    *reinterpret_cast<u32x4_t*>(panel_a(s) + r * kRowBytes + swz(r, c) * 16) = gr[i];
  };
  // codes: thread t takes one 16-value chunk of rows xrow + kXRows i
  const int xrow = t / G::kXChunks, xchunk = t % G::kXChunks;
  const int64_t xcol = k0 + 16 * xchunk;
  uint32_t xoff[kT], soff[kT];
#pragma unroll
  for (int i = 0; i < kT; ++i) {
    const int r = xrow + G::kXRows * i;
    xoff[i] = xcol < k ? (uint32_t)(r * k + xcol) : kOutside;
    soff[i] = xcol < k ? (uint32_t)(r * kb + (xcol >> 5)) : kOutside;
  }
  u32x4_t xc[kT];
  uint32_t xs[kT];
  auto load_x = [&](int64_t s, int i) {
    if constexpr (kGy != kGather) {
      xc[i] = __builtin_amdgcn_raw_buffer_load_b128(rsrc_of(codes + s * kStep * k, step_bytes(s, k)), (int)xoff[i], 0, 0);
      xs[i] = __builtin_amdgcn_raw_buffer_load_b8(rsrc_of(scales + s * kStep * kb, step_bytes(s, kb)), (int)soff[i], 0, 0);
    } else {
      const int64_t row = s * kStep + xrow + G::kXRows * i;
      const bool in = s < s_end && row < m && xcol < k;
      xc[i] = in ? *reinterpret_cast<const u32x4_t*>(codes + row * k + xcol) : u32x4_t{0, 0, 0, 0};
      xs[i] = in ? scales[row * kb + (xcol >> 5)] : 0u;
    }
  };
  auto store_x = [&](int64_t s, int i) {
    uint8_t* dst = panel_b(s);
    const int r = xrow + G::kXRows * i, c = 2 * xchunk;
    uint4 o[2];
    expand16(xc[i], pow2f((int)xs[i] - 127), o);
    *reinterpret_cast<uint4*>(dst + r * kRowBytes + swz_x(r, c) * 16) = o[0];
    *reinterpret_cast<uint4*>(dst + r * kRowBytes + swz_x(r, c + 1) * 16) = o[1];
  };

  // Fragment reads.  The 16 lanes of a group together address four rows of 16 columns (lane
  // j: row j / 4, columns 4 (j % 4) ..) and receive one column each: lane j column j, the
  // four rows in order.  An MFMA lane l holds column l % 32 and rows 8 (l / 32) .. + 7 of
  // the 16-row sub-step: two reads.  Row % 4 is (l % 16) / 4 for every read of a lane.
  const int q = (lane & 15) >> 2;
  const int lrow = 8 * (lane >> 5) + q;
  const int lbyte = lrow * kRowBytes + 32 * ((lane >> 4) & 1) + 8 * (lane & 3);
  // Column tile ti of the panel holds chunks 4 ti ..; those of x sit one off where bit 3 of
  // the chunk, bit 1 of ti, is set.
  auto fragment = [&](const uint8_t* panel, int ti, int sub, int flip) {
    const uint8_t* p = panel + (lbyte ^ (flip << 4)) + ((ti ^ q) << 6) + sub * 16 * kRowBytes;
    const short4_t lo = read_tr(p), hi = read_tr(p + 4 * kRowBytes);
    return __builtin_bit_cast(bf16x8_t, (short8_t){lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]});
  };

  float16_t acc[kT][kT];
#pragma unroll
  for (int i = 0; i < kT; ++i)
#pragma unroll
    for (int j = 0; j < kT; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;

  auto load_fragments = [&](int64_t s, int sub, int i, bf16x8_t (&fa)[kT], bf16x8_t (&fb)[kT]) {
    fa[i] = fragment(panel_a(s), kT * wn + i, sub, 0);
    fb[i] = fragment(panel_b(s), kT * wk + i, sub, ((kT * wk + i) >> 1) & 1);
  };
  // One sub-step: the MFMAs of fragments fa, fb in kT groups; group i first does fill(i) and
  // loads part i of the fragments of sub-step `sub` of step s.
  auto sub_step = [&](const bf16x8_t (&fa)[kT], const bf16x8_t (&fb)[kT], int64_t s, int sub, bf16x8_t (&next_a)[kT],
                      bf16x8_t (&next_b)[kT], auto fill) {
#pragma unroll
    for (int i = 0; i < kT; ++i) {
      fill(i);
      load_fragments(s, sub, i, next_a, next_b);
#pragma unroll
      for (int j = 0; j < kT; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fb[j], fa[i], acc[i][j], 0, 0, 0);
      interleave<kT, 4 / kT>();
    }
  };

  // Four sub-steps of 16 rows per step; each reads the fragments of the next while its own
  // MFMAs run.  The barrier stands before the last: by then this step's panels are read
  // (their last fragments are in registers) and the next step's are complete, so the copies
  // of the step after that start into the freed panels.
  //
  // Codes are loaded, and gy is copied, about a step before they are waited for.  The one
  // wait for both stands in the middle of the third sub-step, as late as the LDS writes of
  // the expanded codes allow, and each load is issued between two groups of MFMAs.  (4096
  // rows, 25600 x 5120: with the wait in the second sub-step and all loads together behind
  // the barrier 960 us, so 897; of zeros, where the clock does not fall under the power of
  // the MFMAs, 890 and 766.)
  constexpr int kMid = kT / 2;
  const auto nothing = [](int) {};
  bf16x8_t fa[2][kT], fb[2][kT];
  // a step's gy into its panel, or (kLoad) into registers
  auto fetch_gy = [&](int64_t s) {
#pragma unroll
    for (int i = 0; i < 2 * kT; ++i) {
      if constexpr (kGy == kLoad) load_gy(s, i);
      else stage_gy(s, i);
    }
  };
#pragma unroll
  for (int i = 0; i < kT; ++i) load_x(s_begin, i);
  fetch_gy(s_begin);
#pragma unroll
  for (int i = 0; i < kT; ++i) store_x(s_begin, i);
  if constexpr (kGy == kLoad) {
    trim_gy(s_begin);
#pragma unroll
    for (int i = 0; i < 2 * kT; ++i) store_gy(s_begin, i);
  }
#pragma unroll
  for (int i = 0; i < kT; ++i) load_x(s_begin + 1, i);
  fetch_gy(s_begin + 1);
  step_barrier();
#pragma unroll
  for (int i = 0; i < kT; ++i) load_fragments(s_begin, 0, i, fa[0], fb[0]);
#pragma clang loop unroll(disable)
  for (int64_t s = s_begin; s < s_end; ++s) {
    sub_step(fa[0], fb[0], s, 1, fa[1], fb[1], nothing);
    sub_step(fa[1], fb[1], s, 2, fa[0], fb[0], nothing);
    sub_step(fa[0], fb[0], s, 3, fa[1], fb[1], [&](int i) {
      if (i < kMid) return;
      if (i == kMid) {
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        if constexpr (kGy == kLoad) trim_gy(s + 1);
      }
      const int h = i - kMid;
#pragma unroll
      for (int j = 2 * h; j < 2 * h + 2; ++j) store_x(s + 1, j);
      if constexpr (kGy == kLoad)
#pragma unroll
        for (int j = 4 * h; j < 4 * h + 4; ++j) store_gy(s + 1, j);
#pragma unroll
      for (int j = 2 * h; j < 2 * h + 2; ++j) load_x(s + 2, j);
    });
    panel_barrier();
    sub_step(fa[1], fb[1], s + 1, 0, fa[0], fb[0], [&](int i) {
      if constexpr (kGy == kLoad) {
        load_gy(s + 2, i);
        load_gy(s + 2, kT + i);
      } else {
        stage_gy(s + 2, i);
        stage_gy(s + 2, kT + i);
      }
    });
  }
  step_barrier();   // no copy still landing in LDS

  // The product is computed transposed (x as the first operand): entry e of lane l is
  // column 8 (e / 4) + 4 (l / 32) + e % 4 of row l % 32, so a lane holds runs of four
  // columns.  32 rows at a time pass through the wave's own LDS region (a row stride of 4
  // words past a multiple of 32 keeps eight rows in different banks) and leave row by row.
  float* st = reinterpret_cast<float*>(lds) + wave * 32 * G::kOutRow;
  const int64_t orow0 = n0 + wn * 32 * kT, ocol0 = k0 + wk * 32 * kT;
#pragma unroll
  for (int i = 0; i < kT; ++i) {
#pragma unroll
    for (int j = 0; j < kT; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        *reinterpret_cast<float4*>(st + (lane & 31) * G::kOutRow + 32 * j + 8 * e + 4 * (lane >> 5)) =
            make_float4(acc[i][j][4 * e], acc[i][j][4 * e + 1], acc[i][j][4 * e + 2], acc[i][j][4 * e + 3]);
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    if (kOutBf16 && splits == 1) {
      constexpr int kLanes = 4 * kT;   // lanes per row, 8 values each
      const int64_t col = ocol0 + 8 * (lane % kLanes);
#pragma unroll
      for (int p = 0; p < 32 * kLanes / 64; ++p) {
        const int r = 64 / kLanes * p + lane / kLanes;
        const float4* f = reinterpret_cast<const float4*>(st + r * G::kOutRow + 8 * (lane % kLanes));
        const float4 a = f[0], b = f[1];
        const int64_t row = orow0 + 32 * i + r;
        if (row < n && col < k)
          __builtin_nontemporal_store(u32x4_t{gemm::pack_bf16x2(a.x, a.y), gemm::pack_bf16x2(a.z, a.w),
                                              gemm::pack_bf16x2(b.x, b.y), gemm::pack_bf16x2(b.z, b.w)},
                                      reinterpret_cast<u32x4_t*>(static_cast<uint16_t*>(out) + row * k + col));
      }
    } else {
      constexpr int kLanes = 8 * kT;   // lanes per row, 4 values each
      float* dst = splits > 1 ? partial + (int64_t)split * n * k : static_cast<float*>(out);
      const int64_t col = ocol0 + 4 * (lane % kLanes);
#pragma unroll
      for (int p = 0; p < 32 * kLanes / 64; ++p) {
        const int r = 64 / kLanes * p + lane / kLanes;
        const u32x4_t v = *reinterpret_cast<const u32x4_t*>(st + r * G::kOutRow + 4 * (lane % kLanes));
        const int64_t row = orow0 + 32 * i + r;
        if (row < n && col < k) {
          // partials are read again at once, the result is not
          u32x4_t* d = reinterpret_cast<u32x4_t*>(dst + row * k + col);
          if (splits > 1) *d = v;
          else __builtin_nontemporal_store(v, d);
        }
      }
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  }
}

// Adds the partials [splits][count] in split order, four values per thread (k is a
// multiple of 16, so count is one of 4).
template <bool kOutBf16>
__global__ void __launch_bounds__(256) weight_grad_reduce(const float* __restrict__ partial, int splits, int64_t count,
                                                          void* __restrict__ out) {
  const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
  if (i >= count) return;
  float4 a = *reinterpret_cast<const float4*>(partial + i);
  for (int s = 1; s < splits; ++s) {
    const float4 b = *reinterpret_cast<const float4*>(partial + s * count + i);
    a.x += b.x;
    a.y += b.y;
    a.z += b.z;
    a.w += b.w;
  }
  if (kOutBf16)
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(out) + i) =
        make_uint2(gemm::pack_bf16x2(a.x, a.y), gemm::pack_bf16x2(a.z, a.w));
  else
    *reinterpret_cast<float4*>(static_cast<float*>(out) + i) = a;
}

// Tile size and row splits.
//
// A round of large tiles (one per compute unit) takes about 5/3 of a round of small ones
// (two per compute unit, half the work), so the sizes are weighed by their whole rounds
// (measured, 4096 rows, large against small: 5120 x 5120, 2 rounds against 4, 200 us against
// 232; 3328 x 5120, 2 against 3, 198 against 173; 8192 x 5120, 3 against 5, 311 against 350;
// 777 rows, 1024 x 5120, 1 against 1, 29 against 19).
//
// A small tile's rows are split across workgroups while there are fewer tiles than compute
// units, each split four steps long at least: the partials (4 bytes a value and split,
// written and read again) cost more than idle slots beyond that (777 rows, 1024 x 5120, 320
// tiles: unsplit 19 us, two ways 31; 4096 rows, 64 x 5120, 40 tiles: unsplit 41, six ways
// 16.3, twelve 18).  Splits that stay 32 steps long fill the second slot of each compute
// unit too (16384 rows, 1024 x 1024: four ways 51 us, eight 46.5).
struct Plan {
  int t, splits;
};
int64_t tiles_of(int64_t n, int64_t k, int tile) { return ((n + tile - 1) / tile) * ((k + tile - 1) / tile); }
Plan plan_of(int64_t m, int64_t n, int64_t k, int cus) {
  const int64_t tiles = tiles_of(n, k, Geo<2>::kTile);
  const int64_t large_rounds = (tiles_of(n, k, Geo<4>::kTile) + cus - 1) / cus;
  const int64_t small_rounds = (tiles + 2 * cus - 1) / (2 * cus);
  if (5 * large_rounds <= 3 * small_rounds) return {4, 1};
  const int64_t steps = (m + kStep - 1) / kStep;
  int64_t sp = std::min<int64_t>(cus / tiles, steps / 4);
  const int64_t twice = 2 * cus / tiles;
  if (steps >= 32 * twice) sp = twice;
  return {2, (int)std::max<int64_t>(sp, 1)};
}

template <int kT, Gy kGy, bool kOutBf16>
hipError_t launch_t(const uint16_t* gy, int64_t m, int64_t n, const uint8_t* codes, const uint8_t* scales, int64_t k,
                    void* grad_w, int splits, float* partial, hipStream_t s) {
  constexpr int kTile = Geo<kT>::kTile, kLds = Geo<kT>::kLds;
  static bool attr_set[kMaxDevices] = {};
  if (hipError_t e = set_dynamic_lds_once(reinterpret_cast<const void*>(&weight_grad_kernel<kT, kGy, kOutBf16>), kLds,
                                          attr_set);
      e != hipSuccess)
    return e;
  const int tn = (int)((n + kTile - 1) / kTile), tk = (int)((k + kTile - 1) / kTile);
  hipLaunchKernelGGL((weight_grad_kernel<kT, kGy, kOutBf16>), dim3((uint32_t)((int64_t)tn * tk * splits)), dim3(256),
                     kLds, s, gy, m, n, codes, scales, k, grad_w, tn, tk, splits, partial);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || splits == 1) return e;
  const int64_t count = n * k;
  hipLaunchKernelGGL((weight_grad_reduce<kOutBf16>), dim3((uint32_t)((count / 4 + 255) / 256)), dim3(256), 0, s,
                     partial, splits, count, grad_w);
  return hipGetLastError();
}

}  // namespace

size_t weight_grad_workspace_bytes(int64_t m, int64_t n, int64_t k, int cus) {
  const int sp = plan_of(m, n, k, cus).splits;
  return sp > 1 ? (size_t)sp * (size_t)n * (size_t)k * sizeof(float) : 0;
}

hipError_t launch_weight_grad(const uint16_t* gy, int64_t m, int64_t n, const uint8_t* codes, const uint8_t* scales,
                              int64_t k, void* grad_w, bool out_bf16, void* workspace, size_t workspace_bytes,
                              int cus, hipStream_t s) {
  Plan p = plan_of(m, n, k, cus);
  if (p.splits > 1 && (workspace == nullptr || workspace_bytes < weight_grad_workspace_bytes(m, n, k, cus))) p.splits = 1;
  float* partial = p.splits > 1 ? static_cast<float*>(workspace) : nullptr;
  using Fn = decltype(&launch_t<4, kCopy, false>);
  static constexpr Fn f[2][3][2] = {{{launch_t<2, kCopy, false>, launch_t<2, kCopy, true>},
                                     {launch_t<2, kLoad, false>, launch_t<2, kLoad, true>},
                                     {launch_t<2, kGather, false>, launch_t<2, kGather, true>}},
                                    {{launch_t<4, kCopy, false>, launch_t<4, kCopy, true>},
                                     {launch_t<4, kLoad, false>, launch_t<4, kLoad, true>},
                                     {launch_t<4, kGather, false>, launch_t<4, kGather, true>}}};
  const Gy how = m == 0 || n < 8 || n >= kBufferWidth || k >= kBufferWidth ? kGather : n % 8 == 0 ? kCopy : kLoad;
  return f[p.t == 4 ? 1 : 0][how][out_bf16 ? 1 : 0](gy, m, n, codes, scales, k, grad_w, p.splits, partial, s);
}

}  // namespace nvfp4
