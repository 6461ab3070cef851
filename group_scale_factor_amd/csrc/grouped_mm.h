// The grouped products of 8-bit operands on gfx950's matrix cores, shared by the
// MXFP8 entry points (E8M0 scale per 32) and the block-128 ones (binary32 scale).
//
// Every product is D[token, n] = sum_k t[token, k] w[n, k] of two row-major code
// matrices, k running along both rows:
//   rows   (M groups): t = a group's activation rows, w = its expert's weights
//   depth  (K groups): t = M features, w = N features, k = the group's tokens
// A Job holds one output tile's operands; make_job finds it from the device end
// offsets, so no launch waits for a group size.
//
// v_mfma_scale_f32_16x16x128_f8f6f4 multiplies 16 rows of w by 16 of t over 128
// elements of k: w goes in as its row operand, t as its column operand, so a lane
// holds one token (lane & 15) and four neighbouring n ((lane >> 4)*4 ..+3) and a
// token's outputs leave side by side. A lane's operand is two 16-byte pieces,
// k = 16*(lane >> 4).. and 64 + 16*(lane >> 4)..; it gives the E8M0 scale of its
// row (lane & 15) for block lane >> 4 of 32 (measured on the card: the scale of
// lane group b applies to k in [32b, 32b + 32)).
//   MX: the four scale bytes of a row and step are one word of the blocked
//       layout; each lane shifts its byte down. No other work on the scales.
//   128: the step is exactly one block, so its sum is formed from zero with scale
//       1 and added to the total times the two blocks' scales (one fma an output). The
//       largest tiles over tokens put scales that are powers of two into the product.
#pragma once

#include <hip/hip_runtime.h>
#include <limits.h>
#include <math.h>
#include <stdint.h>

#include <type_traits>

#include "group_table.h"
#include "launch_order.h"
#include "mx_rearrange.h"

namespace {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef __bf16 v4bf __attribute__((ext_vector_type(4)));

constexpr int kStep = 128;                    // bytes of k per matrix instruction
constexpr int kTileBytes = 512;               // one 128 x 4 tile of blocked scales
constexpr uint32_t kAnyBytes = 0x80000000u;   // buffer size above every valid offset, below kOutOfRange
constexpr int kUnitScales = 0x7f7f7f7f;       // E8M0 2^0 in every byte
// Both scales the constant 0: the builtin is the instruction without scales, which takes no register for them. (As a
// scale, byte 0 would be 2^-127: a test reads off the assembly that no product is made with one.)
constexpr int kNoScales = 0;

struct MmParams {
  const uint8_t *a, *b;       // codes: t and w of every job
  const void *as, *bs;        // their scales
  const int32_t *offs;
  uint16_t *out;
  int64_t a_ld, b_ld;         // bytes between rows
  int64_t b_group_ld;         // rows: bytes between experts
  int64_t out_ld;             // elements
  int64_t slots;              // rows: row tiles at most; depth: groups * M tiles
  int rows;                   // rows: rows of a; depth: M
  int N;
  int K;                      // rows: K; depth: tokens (T, or padded tokens)
  int T;                      // depth: range of the token offsets
  int groups;
  int n_tiles;
  int m_tiles;                // depth: M tiles
};

// One output tile. Everything is the same for the whole workgroup. What K = 0 leaves alone stays as it was, so a Job
// starts as zeros: the paired kernel issues the loads of such a tile, too, out of range of buffers that are none.
struct Job {
  const uint8_t *t, *w;       // first row of the tile, first k
  int t_rows, w_rows;         // valid rows from there
  int K;                      // 0: the tile's outputs are zero
  // MX: blocked matrices from the 128-row block of the tile's first row; its row within that block
  const uint8_t *ts, *ws;
  uint32_t ts_bytes, ws_bytes;
  int t_at, w_at, tile_cols;
  // 128
  const float *tf, *wf;       // scale of the tile's first row or block, first step
  int64_t tf_ld, wf_ld;       // floats from one step to the next
  uint16_t *out;
};

// Tile `slot` of the row tiles of all groups (`tile` rows each, the last of a
// group shorter), the rows past the last end taken as one more group, -1.
struct RowTile {
  int group, row, rows;       // first row, valid rows from it (0: no such tile)
  int local, size, padded;    // place of `row` in the group, its size, its padded start
};

__device__ __forceinline__ RowTile find_row_tile(const int32_t *offs, int groups, int rows, int tile, int slot) {
  int carry_end = 0, carry_pend = 0, carry_tiles = 0;
  RowTile r = {-1, 0, 0, 0, 0, 0};
  for (int base = 0; base < groups; base += kWave) {
    int e, pend;
    scan_slice(offs, groups, rows, base, carry_end, carry_pend, e, pend);
    const int prev = wave_shift_up(e, carry_end);
    const int tiles = (e - prev + tile - 1) / tile;       // 0 in lanes past the groups: their end is the last one
    const int run = wave_inclusive_sum(tiles);
    const int before = __popcll(__ballot(carry_tiles + run <= slot));
    if (before < kWave) {
      const int start = __builtin_amdgcn_readlane(prev, before);
      const int end = __builtin_amdgcn_readlane(e, before);
      const int first =
          carry_tiles + __builtin_amdgcn_readlane(run, before) - __builtin_amdgcn_readlane(tiles, before);
      r.group = base + before;
      r.local = (slot - first) * tile;
      r.size = end - start;
      r.row = start + r.local;
      r.rows = min(tile, end - r.row);
      const int pad = __builtin_amdgcn_readlane(pend, before);
      r.padded = pad - (r.size + kTileRows - 1) / kTileRows * kTileRows;
      return r;
    }
    carry_end = __builtin_amdgcn_readlane(e, kWave - 1);
    carry_pend = __builtin_amdgcn_readlane(pend, kWave - 1);
    carry_tiles += __builtin_amdgcn_readlane(run, kWave - 1);
  }
  const int64_t row = carry_end + int64_t(slot - carry_tiles) * tile;
  if (row < rows) {
    r.row = int(row);
    r.rows = min(tile, rows - r.row);
  }
  return r;
}

// Row tiles of any group sizes that add up to at most `rows`: every group and the rows in none may end in a part.
inline int64_t row_tiles(int64_t rows, int64_t groups, int tile) {
  return rows / tile + (groups < rows ? groups : rows) + 1;
}

// A depth group: its first column along k and width, and the sum of the padded widths before it, in units of
// `unit` tokens padded to `pad` units (MX: 32 and 4; 128: 1 and 128).
struct DepthGroup {
  int start, width, padded;
};

template <int UNIT, int PAD>
__device__ __forceinline__ DepthGroup find_depth_group(const int32_t *offs, int groups, int T, int group) {
  int carry_end = 0, carry_pad = 0;
  DepthGroup d = {0, 0, 0};
  for (int base = 0; base < groups; base += kWave) {
    const int g = base + int(threadIdx.x & (kWave - 1));
    int e = g < groups ? offs[g] : 0;
    e = min(max(e, 0), T) / UNIT;
    e = max(wave_inclusive_max(e), carry_end);
    const int prev = wave_shift_up(e, carry_end);
    const int pad = (e - prev + PAD - 1) / PAD * PAD;
    const int run = wave_inclusive_sum(pad) + carry_pad;
    if (group < base + kWave) {
      const int l = group - base;
      d.start = __builtin_amdgcn_readlane(prev, l);
      d.width = __builtin_amdgcn_readlane(e, l) - d.start;
      d.padded = __builtin_amdgcn_readlane(run, l) - __builtin_amdgcn_readlane(pad, l);
      return d;
    }
    carry_end = __builtin_amdgcn_readlane(e, kWave - 1);
    carry_pad = __builtin_amdgcn_readlane(run, kWave - 1);
  }
  return d;
}

__device__ __forceinline__ uint32_t block_bytes_from(int64_t blocks, int tile_cols, int tile) {
  // as many 128-row blocks as one output tile can touch
  const int64_t most = tile / kTileRows + 1;
  return uint32_t((blocks < most ? blocks : most) * tile_cols * kTileBytes);
}

// The job of tile (slot, n tile): false if there is nothing to write.
template <bool MX, bool DEPTH, int TM, int TN>
__device__ __forceinline__ bool make_job(const MmParams &p, const int32_t *offs, uint32_t slot, int nt, Job &j) {
  const int n0 = nt * TN;
  j.w_rows = min(TN, p.N - n0);
  const int nb = (p.N + kTileRows - 1) / kTileRows;
  if (!DEPTH) {
    const RowTile r = find_row_tile(offs, p.groups, p.rows, TM, int(slot));
    if (r.rows <= 0) return false;
    j.t_rows = r.rows;
    j.out = p.out + int64_t(r.row) * p.out_ld + n0;
    j.K = r.group < 0 ? 0 : p.K;
    if (j.K == 0) return true;
    const int steps = (p.K + kStep - 1) / kStep;
    j.t = p.a + int64_t(r.row) * p.a_ld;
    j.w = p.b + int64_t(r.group) * p.b_group_ld + int64_t(n0) * p.b_ld;
    if (MX) {
      j.tile_cols = steps;
      const int64_t tb = (r.padded + r.local) / kTileRows, wb = n0 / kTileRows;
      j.ts = static_cast<const uint8_t *>(p.as) + tb * steps * kTileBytes;
      j.ts_bytes = block_bytes_from((r.size + kTileRows - 1) / kTileRows - r.local / kTileRows, steps, TM);
      j.t_at = r.local % kTileRows;
      j.ws = static_cast<const uint8_t *>(p.bs) + (int64_t(r.group) * nb + wb) * steps * kTileBytes;
      j.ws_bytes = block_bytes_from(nb - wb, steps, TN);
      j.w_at = n0 % kTileRows;
    } else {
      j.tf = static_cast<const float *>(p.as) + r.row;
      j.tf_ld = p.rows;
      j.wf = static_cast<const float *>(p.bs) + (int64_t(r.group) * nb + n0 / kTileRows) * steps;
      j.wf_ld = 1;
    }
  } else {
    const int g = int(slot / uint32_t(p.m_tiles));
    const int m0 = (int(slot) - g * p.m_tiles) * TM;
    j.t_rows = min(TM, p.rows - m0);
    j.out = p.out + (int64_t(g) * p.rows + m0) * p.out_ld + n0;
    int64_t k0;
    if (MX) {
      const DepthGroup d = find_depth_group<32, 4>(offs, p.groups, p.T, g);
      j.K = d.width * 32;
      k0 = int64_t(d.start) * 32;
      j.tile_cols = (d.width + 3) / 4;
      const int mb = (p.rows + kTileRows - 1) / kTileRows;
      // group matrices follow one another: 128 * blocks rows of d.padded columns lie before this one
      j.ts = static_cast<const uint8_t *>(p.as) + int64_t(mb) * kTileRows * d.padded +
             int64_t(m0 / kTileRows) * j.tile_cols * kTileBytes;
      j.ts_bytes = block_bytes_from(mb - m0 / kTileRows, j.tile_cols, TM);
      j.t_at = m0 % kTileRows;
      j.ws = static_cast<const uint8_t *>(p.bs) + int64_t(nb) * kTileRows * d.padded +
             int64_t(n0 / kTileRows) * j.tile_cols * kTileBytes;
      j.ws_bytes = block_bytes_from(nb - n0 / kTileRows, j.tile_cols, TN);
      j.w_at = n0 % kTileRows;
    } else {
      const DepthGroup d = find_depth_group<1, kStep>(offs, p.groups, p.T, g);
      j.K = (d.width + kStep - 1) / kStep * kStep;    // padding holds code 0
      k0 = d.padded;
      j.tf = static_cast<const float *>(p.as) + (k0 / kStep) * p.rows + m0;
      j.tf_ld = p.rows;
      j.wf = static_cast<const float *>(p.bs) + (k0 / kStep) * p.N + n0;
      j.wf_ld = p.N;
    }
    j.t = p.a + int64_t(m0) * p.a_ld + k0;
    j.w = p.b + int64_t(n0) * p.b_ld + k0;
  }
  return true;
}

// Byte offset of scale row `row` (of the matrix's 128-row blocks) at tile column 0.
__device__ __forceinline__ uint32_t scale_row_offset(int row, int tile_cols) {
  return uint32_t(row / kTileRows) * tile_cols * kTileBytes + (row % 32) * 16 + (row % kTileRows / 32) * 4;
}

__device__ __forceinline__ v8i operand(const uint4 &lo, const uint4 &hi) {
  return v8i{int(lo.x), int(lo.y), int(lo.z), int(lo.w), int(hi.x), int(hi.y), int(hi.z), int(hi.w)};
}

__device__ __forceinline__ v4f mfma(const v8i &w, const v8i &t, const v4f &c, int ws, int ts) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, t, c, 0, 0, 0, ws, 0, ts);
}

__device__ __forceinline__ uint4 load16(__amdgpu_buffer_rsrc_t rsrc, uint32_t off) {
  const auto v = __builtin_amdgcn_raw_buffer_load_b128(rsrc, int(off), 0, 0);
  return make_uint4(v[0], v[1], v[2], v[3]);
}

__device__ __forceinline__ uint32_t load4(__amdgpu_buffer_rsrc_t rsrc, uint32_t off) {
  return __builtin_amdgcn_raw_buffer_load_b32(rsrc, int(off), 0, 0);
}

// Four neighbouring outputs of one token, n .. n+3 of `left` valid ones, at the type's own alignment (memory takes
// one wide store at any address: an output of odd width (39, 530, 1630) left in 137 us value by value).
__device__ __forceinline__ void store4(uint16_t *dst, const v4f &v, int left) {
  const v4bf h = __builtin_convertvector(v, v4bf);
  if (left >= 4) {
    __builtin_memcpy(dst, &h, 8);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < left) reinterpret_cast<__bf16 *>(dst)[i] = h[i];
  }
}

// ------------------------------------------------------------- streamed tiles
//
// Straight from memory to registers, no LDS on the way: a workgroup's four waves
// share one tile of TF*16 tokens by 32 outputs and deal its steps of k among
// themselves, so the longest chain is a quarter of k; the four totals meet in LDS.

constexpr int kStreamWaves = 4;
constexpr int kStreamN = 32;

template <bool MX, bool DEPTH, int TF>
struct StreamStep {
  uint4 t[TF][2], w[2][2];
  uint32_t ts[TF];
  uint32_t ws[2][DEPTH && !MX ? 4 : 1];
};

template <bool MX, bool DEPTH, int TF>
__global__ __launch_bounds__(kStreamWaves *kWave) void mm_stream_kernel(MmParams p) {
  __shared__ v4f totals[kStreamWaves][TF * 2][kWave];
  const uint32_t slot = blockIdx.x / uint32_t(p.n_tiles);
  Job j;
  if (!make_job<MX, DEPTH, TF * 16, kStreamN>(p, p.offs, slot, int(blockIdx.x - slot * p.n_tiles), j)) return;
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x) / kWave);
  const int r = lane & 15, g = lane >> 4;

  v4f acc[TF][2];
#pragma unroll
  for (int i = 0; i < TF; ++i)
#pragma unroll
    for (int n = 0; n < 2; ++n) acc[i][n] = v4f{0, 0, 0, 0};

  if (j.K > 0) {
    const __amdgpu_buffer_rsrc_t tr = byte_buffer(j.t, kAnyBytes), wr = byte_buffer(j.w, kAnyBytes);
    __amdgpu_buffer_rsrc_t tsr, wsr;
    if (MX) {
      tsr = byte_buffer(j.ts, j.ts_bytes);
      wsr = byte_buffer(j.ws, j.ws_bytes);
    }
    const int steps = (j.K + kStep - 1) / kStep;
    const auto fetch = [&](int s, StreamStep<MX, DEPTH, TF> &f) {
      const int k = s * kStep + g * 16;
#pragma unroll
      for (int i = 0; i < TF; ++i) {
        const bool row = i * 16 + r < j.t_rows;
        const uint32_t off = uint32_t((i * 16 + r) * uint32_t(p.a_ld) + k);
        f.t[i][0] = load16(tr, row && k < j.K ? off : kOutOfRange);
        f.t[i][1] = load16(tr, row && k + 64 < j.K ? off + 64 : kOutOfRange);
        if (MX)
          f.ts[i] = load4(tsr, scale_row_offset(j.t_at + i * 16 + r, j.tile_cols) + uint32_t(s) * kTileBytes);
        else
          f.ts[i] = row ? __float_as_uint(j.tf[s * j.tf_ld + i * 16 + r]) : 0u;
      }
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const bool row = n * 16 + r < j.w_rows;
        const uint32_t off = uint32_t((n * 16 + r) * uint32_t(p.b_ld) + k);
        f.w[n][0] = load16(wr, row && k < j.K ? off : kOutOfRange);
        f.w[n][1] = load16(wr, row && k + 64 < j.K ? off + 64 : kOutOfRange);
        if (MX) {
          f.ws[n][0] = load4(wsr, scale_row_offset(j.w_at + n * 16 + r, j.tile_cols) + uint32_t(s) * kTileBytes);
        } else if (DEPTH) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int at = n * 16 + g * 4 + e;
            f.ws[n][DEPTH && !MX ? e : 0] = at < j.w_rows ? __float_as_uint(j.wf[s * j.wf_ld + at]) : 0u;
          }
        } else {
          f.ws[n][0] = __float_as_uint(j.wf[s]);
        }
      }
    };
    const auto multiply = [&](const StreamStep<MX, DEPTH, TF> &f) {
#pragma unroll
      for (int i = 0; i < TF; ++i)
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          const v8i w = operand(f.w[n][0], f.w[n][1]), t = operand(f.t[i][0], f.t[i][1]);
          if (MX) {
            acc[i][n] = mfma(w, t, acc[i][n], int(f.ws[n][0] >> (8 * g)), int(f.ts[i] >> (8 * g)));
          } else {
            const v4f part = mfma(w, t, v4f{0, 0, 0, 0}, kUnitScales, kUnitScales);
            const float ts = __uint_as_float(f.ts[i]);
#pragma unroll
            for (int e = 0; e < 4; ++e)
              acc[i][n][e] = fmaf(part[e], ts * __uint_as_float(f.ws[n][DEPTH && !MX ? e : 0]), acc[i][n][e]);
          }
        }
    };
    StreamStep<MX, DEPTH, TF> now, next;
    if (wave < steps) fetch(wave, now);
    for (int s = wave; s < steps; s += kStreamWaves) {
      if (s + kStreamWaves < steps) fetch(s + kStreamWaves, next);
      multiply(now);
      now = next;
    }
  }
#pragma unroll
  for (int i = 0; i < TF; ++i)
#pragma unroll
    for (int n = 0; n < 2; ++n) totals[wave][i * 2 + n][lane] = acc[i][n];
  __syncthreads();
  for (int at = int(threadIdx.x); at < TF * 2 * kWave; at += kStreamWaves * kWave) {
    const int f = at / kWave, l = at % kWave;
    const int token = f / 2 * 16 + (l & 15), n = f % 2 * 16 + (l >> 4) * 4;
    v4f sum = totals[0][f][l];
#pragma unroll
    for (int w = 1; w < kStreamWaves; ++w) sum += totals[w][f][l];
    if (token < j.t_rows && n < j.w_rows) store4(j.out + int64_t(token) * p.out_ld + n, sum, j.w_rows - n);
  }
}

// ------------------------------------------------------------- staged tiles
//
// TW x NW waves share a tile of TW*TF*16 tokens by NW*64 outputs. Each step's
// 128 bytes of every row, and its scales, go straight from memory to LDS (buffer
// loads with an LDS destination), STAGES - 1 steps ahead of the products.
// A row is eight 16-byte pieces; piece c of row r sits at place c ^ key(r), so
// that the 16 rows x 4 pieces a wave reads at once cover every bank evenly:
// key(r) = r mod 8 for t; for w, whose fragment j takes rows 32*(j/2) + 8*(r/4) +
// 4*(j%2) + r%4 (a lane then ends up with twice eight neighbouring outputs of its
// token, four lanes with 64 bytes), the same three bits of that row's place in the
// fragment. The load puts them there: its LDS side is lane-linear, so the lane's
// memory address carries the permutation.

typedef uint32_t v4u __attribute__((ext_vector_type(4)));

// BYTES (16 or 4) a lane from memory to LDS (the wave's 64 * BYTES from `lds` on, lane by lane). The compiler does
// not see this load: it orders nothing after it and waits for it nowhere, so a product may read one stage while the
// other fills; wait_loads() before the barrier is what completes it. Lanes out of range write zeros.
// `skip` (uniform) is added to every lane's offset; the range check counts it (measured: zeros from the buffer's end
// on for offset + skip, also where offset + skip passes 2^32 or skip alone the size). m0 is declared as written: the
// compiler reserves it, warns of that, and makes it anew wherever it needs it itself (which is nowhere here).
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
template <int BYTES>
__device__ __forceinline__ void load_to_lds(const v4u &rsrc, uint32_t lds, uint32_t off, uint32_t skip = 0) {
  if (BYTES == 16)
    asm volatile(
        "s_mov_b32 m0, %0\n\t"
        "s_nop 0\n\t"
        "buffer_load_dwordx4 %1, %2, %3 offen lds"
        :
        : "s"(lds), "v"(off), "s"(rsrc), "s"(skip)
        : "m0", "memory");
  else
    asm volatile(
        "s_mov_b32 m0, %0\n\t"
        "s_nop 0\n\t"
        "buffer_load_dword %1, %2, %3 offen lds"
        :
        : "s"(lds), "v"(off), "s"(rsrc), "s"(skip)
        : "m0", "memory");
}
#pragma clang diagnostic pop

// All but the newest LEFT loads of this wave are complete; with READS its reads of LDS, too: a barrier behind which
// others write there stands behind them by itself, not by where the compiler puts the products that use them.
template <int LEFT, bool READS = false>
__device__ __forceinline__ void wait_loads() {
  static_assert(LEFT < 64, "six bits of the count: 0..3 and 14, 15");
  __builtin_amdgcn_s_waitcnt((READS ? 0x0070 : 0x0f70) | (LEFT & 15) | (LEFT >> 4 << 14));
}

__device__ __forceinline__ v4u raw_buffer(const void *base, uint32_t bytes) {
  const uint64_t a = reinterpret_cast<uint64_t>(base);
  return v4u{uint32_t(__builtin_amdgcn_readfirstlane(int(uint32_t(a)))),
             uint32_t(__builtin_amdgcn_readfirstlane(int(uint32_t(a >> 32)))) & 0xffffu,
             uint32_t(__builtin_amdgcn_readfirstlane(int(bytes))), uint32_t(kRawBufferFlags)};
}

// First row of fragment n of w, from the lane's.
__device__ constexpr int w_row(int n) { return (n >> 1) * 32 + (n & 1) * 4; }

constexpr int kBand = 4;      // row tiles whose n tiles are interleaved: their weights are read together
constexpr int kDeal = 32;     // neighbouring tiles dealt to one XCD (one for each of its CUs)

// The LDS of a staged tile: STAGES stages of codes, then as many of scales (in loads of 256 bytes: 64 words).
template <bool MX, bool DEPTH, int TW, int NW, int TF, int STAGES_>
struct TileShape {
  static constexpr int TM = TW * TF * 16, TN = NW * 64, WAVES = TW * NW, STAGES = STAGES_;
  static constexpr int TBytes = TM * kStep, Stage = TBytes + TN * kStep;
  static constexpr int TQ = TM / 8 / WAVES, WQ = TN / 8 / WAVES;     // loads of eight rows per wave and step
  static constexpr int TS = MX ? 2 * ((TM + kTileRows - 1) / kTileRows) : (TM + 63) / 64;      // loads of t's scales
  static constexpr int WS = MX ? 2 * (TN / kTileRows) : DEPTH ? TN / 64 : 1;
  static constexpr int SQ = (TS + WS + WAVES - 1) / WAVES;           // scale loads per wave and step
  static constexpr int Loads = TQ + WQ + SQ;                         // of a wave and step
  static constexpr int Scales = STAGES * Stage, ScaleStage = (SQ * WAVES + 1) * 256;
  static constexpr int Lds = Scales + STAGES * ScaleStage;
};

// A wave's outputs, TF*16 tokens from t_first by 64 from n_first on, by way of 2 KB of LDS of its own: a lane has 16
// bytes here and there of 16 rows, and 64 bytes of each of them take the address unit 33 cycles a store; eight
// whole 128-byte rows take it 11 (a 256 x 256 tile: 4170 cycles and 1450). The 16-byte pieces of a row are XOR-ed by
// its number as the staged ones are. LDS works in order, so a fragment's pieces follow the reads of the one before.
// With FULL every row and column is valid: TF * 2 stores of every lane.
template <int TF, bool FULL>
__device__ __forceinline__ void store_rows(uint16_t *out, int64_t out_ld, int t_rows, int w_rows,
                                           const v4f (&acc)[TF][4], uint8_t *lds, int t_first, int n_first) {
  typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
  int lane = threadIdx.x & (kWave - 1);
  asm volatile("" : "+v"(lane), "+s"(t_first), "+s"(n_first), "+s"(out_ld));      // nothing made from these waits in
                                                                                  // a register for a tile's end
  const int r = lane & 15, g = lane >> 4;
  const int left = w_rows - n_first - (lane & 7) * 8;
  uint16_t *dst = out + int64_t(t_first + (lane >> 3)) * out_ld + n_first + (lane & 7) * 8;
#pragma unroll
  for (int i = 0; i < TF; ++i) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const v4bf a = __builtin_convertvector(acc[i][2 * h], v4bf);
      const v4bf b = __builtin_convertvector(acc[i][2 * h + 1], v4bf);
      *reinterpret_cast<v8bf *>(lds + r * 128 + ((h * 4 + g) ^ (r & 7)) * 16) =
          __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
    }
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int row = q * 8 + (lane >> 3);
      const v8bf v = *reinterpret_cast<const v8bf *>(lds + row * 128 + ((lane & 7) ^ (row & 7)) * 16);
      uint16_t *to = dst + int64_t(i * 16 + q * 8) * out_ld;
      if (FULL) {
        __builtin_memcpy(to, &v, 16);
      } else if (t_first + i * 16 + row < t_rows) {
        if (left >= 8) {
          __builtin_memcpy(to, &v, 16);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (e < left) reinterpret_cast<__bf16 *>(to)[e] = v[e];
        }
      }
    }
  }
}

// Tile of workgroup `block`: runs of kDeal tiles dealt to the XCDs in turn (workgroup b runs on XCD b mod 8), bands of
// kBand row tiles with their n tiles interleaved. 32-bit arithmetic: a grid holds fewer than 2^32 / threads
// workgroups, and 64-bit divisions took a workgroup 1 us.
struct TilePlace {
  uint32_t slot, n;
};

__device__ __forceinline__ bool place_tile(const MmParams &p, uint32_t block, TilePlace &t) {
  const uint32_t slots = uint32_t(p.slots), n_tiles = uint32_t(p.n_tiles);
  const uint32_t k = block / 8;
  const uint32_t unit = ((k / kDeal) * 8 + block % 8) * kDeal + k % kDeal;
  if (unit >= slots * n_tiles) return false;
  const uint32_t band = unit / (kBand * n_tiles);
  const uint32_t at = unit - band * kBand * n_tiles;
  const uint32_t in_band = min(slots - band * kBand, uint32_t(kBand));
  t.n = in_band == kBand ? at / kBand : at / in_band;
  t.slot = band * kBand + (at - t.n * in_band);
  return true;
}

template <bool MX, bool DEPTH, int TW, int NW, int TF, int STAGES>
__global__ __launch_bounds__(TW *NW *kWave) void mm_tile_kernel(MmParams p) {
  using S = TileShape<MX, DEPTH, TW, NW, TF, STAGES>;
  extern __shared__ __align__(1024) uint8_t mm_lds[];
  TilePlace at;
  if (!place_tile(p, blockIdx.x, at)) return;
  Job j;
  if (!make_job<MX, DEPTH, S::TM, S::TN>(p, p.offs, at.slot, int(at.n), j)) return;

  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x) / kWave);
  const int tw = wave / NW, nw = wave % NW;
  const int r = lane & 15, g = lane >> 4;
  const int t_first = tw * TF * 16, n_first = nw * 64;      // the wave's part of the tile

  v4f acc[TF][4];
#pragma unroll
  for (int i = 0; i < TF; ++i)
#pragma unroll
    for (int n = 0; n < 4; ++n) acc[i][n] = v4f{0, 0, 0, 0};

  if (j.K > 0) {
    const uint32_t lds = uint32_t(__builtin_amdgcn_readfirstlane(
        int(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) uint8_t *)mm_lds))));
    const int steps = (j.K + kStep - 1) / kStep;

    // addresses of this lane's pieces: eight rows a load, lane / 8 the row, lane % 8 the place
    uint32_t toff[S::TQ], woff[S::WQ];
    int tk, wk[2];     // the piece's place along k
    tk = ((lane & 7) ^ (lane >> 3)) * 16;
#pragma unroll
    for (int q = 0; q < S::TQ; ++q) {
      const int row = (wave * S::TQ + q) * 8 + (lane >> 3);
      toff[q] = row < j.t_rows ? uint32_t(row) * uint32_t(p.a_ld) + tk : kOutOfRange;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) wk[h] = ((lane & 7) ^ (((lane >> 3) & 3) | (h << 2))) * 16;
#pragma unroll
    for (int q = 0; q < S::WQ; ++q) {
      const int row = (wave * S::WQ + q) * 8 + (lane >> 3);
      const int k = wk[(wave * S::WQ + q) & 1];
      woff[q] = row < j.w_rows ? uint32_t(row) * uint32_t(p.b_ld) + k : kOutOfRange;
    }
    const auto stage = [&](int s) {
      const uint32_t place = uint32_t(s) % STAGES;
      const uint32_t base = lds + place * S::Stage;
      const uint32_t to = base + wave * S::TQ * 1024, tow = base + S::TBytes + wave * S::WQ * 1024;
      const int k0 = s * kStep;
      const v4u tr = raw_buffer(j.t + k0, kAnyBytes), wr = raw_buffer(j.w + k0, kAnyBytes);
#pragma unroll
      for (int q = 0; q < S::SQ; ++q) {
        const int at = wave + q * S::WAVES;              // which 64 scale words
        const bool t = at < S::TS;
        const int word = (t ? at : at - S::TS) * 64 + lane;
        const uint32_t dst = lds + S::Scales + place * S::ScaleStage + at * 256;
        if (MX) {
          // two loads for each 128 x 4 tile; the next tile of rows lies tile_cols tiles on
          const uint32_t off = uint32_t(word / 128 * j.tile_cols + s) * kTileBytes + word % 128 * 4;
          load_to_lds<4>(raw_buffer(t ? j.ts : j.ws, t ? j.ts_bytes : j.ws_bytes), dst,
                         at < S::TS + S::WS && s < steps ? off : kOutOfRange);
        } else if (t || DEPTH) {
          const int rows = t ? j.t_rows : j.w_rows;
          load_to_lds<4>(raw_buffer(t ? j.tf + s * j.tf_ld : j.wf + s * j.wf_ld, uint32_t(rows) * 4), dst,
                         at < S::TS + S::WS && s < steps ? uint32_t(word) * 4 : kOutOfRange);
        } else {
          // one word for each 128 outputs
          const int per = (p.K + kStep - 1) / kStep;
          load_to_lds<4>(raw_buffer(j.wf + s, kAnyBytes), dst,
                         at == S::TS && s < steps && word * kTileRows < j.w_rows ? uint32_t(word * per) * 4 : kOutOfRange);
        }
      }
      if (k0 + kStep <= j.K) {
#pragma unroll
        for (int q = 0; q < S::TQ; ++q) load_to_lds<16>(tr, to + q * 1024, toff[q]);
#pragma unroll
        for (int q = 0; q < S::WQ; ++q) load_to_lds<16>(wr, tow + q * 1024, woff[q]);
      } else {      // pieces past K are zeros; all of them past the last step (the counts of loads under way stay)
        const int left = j.K - k0;
#pragma unroll
        for (int q = 0; q < S::TQ; ++q) load_to_lds<16>(tr, to + q * 1024, tk < left ? toff[q] : kOutOfRange);
#pragma unroll
        for (int q = 0; q < S::WQ; ++q)
          load_to_lds<16>(wr, tow + q * 1024, wk[(wave * S::WQ + q) & 1] < left ? woff[q] : kOutOfRange);
      }
    };

    const uint32_t t_read = (t_first + r) * kStep + ((g ^ (r & 7)) * 16);
    const uint32_t w_read = S::TBytes + (n_first + (r >> 2) * 8 + (r & 3)) * kStep + ((g ^ (r & 7)) * 16);
    const uint32_t ts_read = S::Scales + (MX ? scale_row_offset(j.t_at + t_first + r, 1) : uint32_t(t_first + r) * 4);
    const uint32_t ws_read = S::Scales + S::TS * 256 +
                             (MX      ? scale_row_offset(n_first + (r >> 2) * 8 + (r & 3), 1)
                              : DEPTH ? uint32_t(n_first + g * 8) * 4
                                      : uint32_t(n_first / kTileRows) * 4);
    const auto multiply = [&](int s) {
      const uint8_t *from = mm_lds + uint32_t(s) % STAGES * S::Stage;
      const uint8_t *scales = mm_lds + uint32_t(s) % STAGES * S::ScaleStage;
      uint32_t ts[TF], ws[MX ? 4 : DEPTH ? 16 : 1];
      if (MX) {
        // rows r, r+32, .. of a 128-row block share 16 bytes, rows r+16, .. the ones 256 bytes on
#pragma unroll
        for (int i = 0; i < TF; ++i)
          ts[i] = *reinterpret_cast<const uint32_t *>(scales + ts_read + (i & 1) * 256 + (i >> 1) * 4) >> (8 * g);
#pragma unroll
        for (int n = 0; n < 4; ++n)
          ws[n] = *reinterpret_cast<const uint32_t *>(scales + ws_read + (n & 1) * 64 + (n >> 1) * 4) >> (8 * g);
      } else {
#pragma unroll
        for (int i = 0; i < TF; ++i) ts[i] = *reinterpret_cast<const uint32_t *>(scales + ts_read + i * 64);
#pragma unroll
        for (int n = 0; n < int(sizeof(ws) / 4); ++n)
          ws[n] = *reinterpret_cast<const uint32_t *>(scales + ws_read + (n / 8 * 32 + n % 8) * 4);
      }
      v8i w[4];
#pragma unroll
      for (int n = 0; n < 4; ++n)
        w[n] = operand(*reinterpret_cast<const uint4 *>(from + w_read + w_row(n) * kStep),
                       *reinterpret_cast<const uint4 *>(from + (w_read ^ 64) + w_row(n) * kStep));
#pragma unroll
      for (int i = 0; i < TF; ++i) {
        const v8i t = operand(*reinterpret_cast<const uint4 *>(from + t_read + i * 16 * kStep),
                              *reinterpret_cast<const uint4 *>(from + (t_read ^ 64) + i * 16 * kStep));
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          if (MX) {
            acc[i][n] = mfma(w[n], t, acc[i][n], int(ws[n]), int(ts[i]));
          } else {
            const v4f part = mfma(w[n], t, v4f{0, 0, 0, 0}, kUnitScales, kUnitScales);
#pragma unroll
            for (int e = 0; e < 4; ++e)
              acc[i][n][e] = fmaf(part[e], __uint_as_float(ts[i]) * __uint_as_float(ws[DEPTH && !MX ? n * 4 + e : 0]),
                                  acc[i][n][e]);
          }
        }
      }
    };

#pragma unroll
    for (int s = 0; s < STAGES - 1; ++s) stage(s);
    for (int s = 0; s < steps; ++s) {
      wait_loads<(STAGES - 2) * S::Loads, true>();      // this wave's part of stage s is in LDS
      __builtin_amdgcn_s_barrier();                     // and everyone's; nobody reads the stage before it any more
      stage(s + STAGES - 1);
      multiply(s);
    }
    wait_loads<0, true>();                        // the out-of-range ones too
    __builtin_amdgcn_s_barrier();                 // nothing is under way into LDS, and nobody reads it any more
    // the products have to be done by the whole wave, before the branches of the stores below
#pragma unroll
    for (int i = 0; i < TF; ++i)
#pragma unroll
      for (int n = 0; n < 4; ++n) asm volatile("" : "+v"(acc[i][n]));
  }

  store_rows<TF, false>(j.out, p.out_ld, j.t_rows, j.w_rows, acc, mm_lds + wave * 2048, t_first, n_first);
}

// ------------------------------------------------------------- paired waves
//
// The 256 x 256 tile of eight waves, two on each SIMD, that take turns: waves 0..3 ("lead", the tokens' first 128
// rows) read their operands of a step from LDS while waves 4..7 (the others) multiply, then the other way round, a
// barrier between the slots:
//   slot       2s       2s+1        2s+2        2s+3
//   lead       read s   multiply s  read s+1    multiply s+1
//   others              read s      multiply s  read s+1
// A wave's operands are w (four fragments of 16 rows, shared with the other group) and eight fragments of t (shared
// within its group). Registers hold four of those: "read" takes w, the scales and the first four (the first half of
// the group's rows), "multiply" replaces each as soon as its products are issued.
//
// A load may go to a place one slot after the place was last read, and has to be there a slot before the next read:
//   w, its scales        last read in slot 2s+1 (others); the next, s+2's, in slot 2s+4 (lead)
//   t, lead              last read in slots 2s, 2s+1; next 2s+4, 2s+5
//   t, others            last read in slots 2s+1, 2s+2; next 2s+5, 2s+6
// A load of 1 KB keeps a wave for 61 cycles where the four waves of a group issue theirs together (64 bytes a cycle
// and CU), and for 240 where it stands between products: all are issued while the group reads, between the LDS
// reads, which then cost nothing on top. lead loads w, its own t and the scales of both (14 loads, about as long as
// the others' 32 products: 1018 cycles), the others their t and its scales.
//
// A workgroup takes tile after tile: the step after a tile's last one is the next tile's first. To find a tile, to wait
// for its first loads (2000 to 5000 cycles from nothing) and to store its outputs (3000) then overlaps with steps,
// which take 3000 cycles each. Against a workgroup for each tile: K groups of 8 steps (16 groups, outputs of 8192 x
// 5120) 852 -> 798 us; row groups of 11 steps (131072 rows, N 5120) 1055 -> 995; of 40 steps the same. From there on
// the card's power sets the rate: 8192 x 8192 x 8192 takes 384 to 440 us on different cards (2.5 to 2.9 PFLOP/s at
// 1.65 to 1.9 GHz).
//
// Block-128 scales multiply a product's sums, and over k that is a multiplication and an addition for each of them
// (each token's and each output's scale): 8 instructions of 4 cycles beside a product's 32, as long as those and on
// the same power. Scales that are powers of two, as the casts give them, go into the products instead, which multiply
// by 2^(byte - 127) anyway: the exponent is the byte. A workgroup takes that for granted, and each wave looks at 64 of
// a step's 512 scales; the first other one ends it, and the workgroup does the tile again, and the ones after it, with
// the multiplications. (Both kinds in one loop write the sums from two places, and 500 registers spill.) Seven groups
// of 32001 tokens, 1408 x 7168: 385 -> 350 us, now 340 to 363; with any scales 8192 x 8192 x 8192 takes 561 us for 555. Row groups
// keep the multiplications: there they are half as many (a step has one scale of w), and weights often have any scales.

template <bool MX, bool DEPTH>
constexpr int paired_lds() {
  return TileShape<MX, DEPTH, 2, 4, 8, 2>::Lds + 8 * 2048 + kWave * 4 + 4;
}

template <bool MX, bool DEPTH>
__global__ __launch_bounds__(512) void mm_paired_kernel(MmParams p) {
  constexpr int NW = 4, TF = 8;
  constexpr bool kChecked = !MX && DEPTH;      // see run() below
  using S = TileShape<MX, DEPTH, 2, NW, TF, 2>;
  static_assert(S::TS == 4 && S::WS <= 4, "scale loads: two for each group's rows of t, up to one a lead wave for w");
  extern __shared__ __align__(1024) uint8_t mm_lds[];
  // LDS behind the stages: 2 KB a wave for its outputs, the end offsets of up to 64 groups, the first step of other
  // scales than powers of two
  constexpr int kOutputs = S::Lds, kEnds = kOutputs + 8 * 2048, kOther = kEnds + kWave * 4;
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x) / kWave);
  const int tw = wave / NW, nw = wave % NW;                 // tw: 0 lead, 1 the others
  const int r = lane & 15, g = lane >> 4;
  const int t_first = tw * TF * 16, n_first = nw * 64;      // the wave's part of the tile

  // The workgroup's tiles: blockIdx.x and every gridDim.x further on that has anything to write. With more than 64
  // groups the grid has a workgroup for each tile.
  uint32_t block = blockIdx.x;
  // Between tiles the arguments are read again: kept in registers, the steps' own scalars would not fit beside them.
  const auto args = [] {
    auto *from = (const __attribute__((address_space(4))) uint8_t *)__builtin_amdgcn_kernarg_segment_ptr();
    asm volatile("" : "+s"(from));
    return (const MmParams *)from;
  };
  const auto find = [&](const int32_t *offs, Job &job) __attribute__((always_inline)) {
    TilePlace at;
    for (; place_tile(*args(), block, at); block += gridDim.x)
      if (make_job<MX, DEPTH, S::TM, S::TN>(*args(), offs, at.slot, int(at.n), job)) {
        block += gridDim.x;
        return true;
      }
    return false;
  };
  Job j = {};      // the tile whose steps are loaded
  if (!find(p.offs, j)) return;
  int32_t *ends = reinterpret_cast<int32_t *>(mm_lds + kEnds);
  if (wave == 0 && p.groups <= kWave && lane < p.groups) ends[lane] = p.offs[lane];
  int *other = reinterpret_cast<int *>(mm_lds + kOther);
  if (kChecked && threadIdx.x == 0) *other = INT_MAX;

  uint16_t *out;              // the tile to multiply: its outputs
  int out_t, out_w;
  v4f acc[TF][4];
  const auto clear = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < TF; ++i)
#pragma unroll
      for (int n = 0; n < 4; ++n) acc[i][n] = v4f{0, 0, 0, 0};
  };

  const uint32_t lds = uint32_t(__builtin_amdgcn_readfirstlane(
      int(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) uint8_t *)mm_lds))));

  // A load takes eight rows: lane / 8 is the row, lane % 8 the place. The buffer of a step starts at its first byte
  // of the tile's first row and holds rows * stride bytes: the row after the last valid one is out of range, and a
  // valid row's own bytes are not. Past the last step the same loads are issued out of range: the counts of loads
  // under way stay the same. (What a load takes beside the four instructions it needs costs here: the reads and
  // loads of a slot are one wave's instructions, one after the other.)
  const int tk = ((lane & 7) ^ (lane >> 3)) * 16;      // the piece's place along k; for w, of even and odd eights
  int wk[2];                                           // of rows
#pragma unroll
  for (int h = 0; h < 2; ++h) wk[h] = ((lane & 7) ^ (((lane >> 3) & 3) | (h << 2))) * 16;
  const uint32_t t_ld = uint32_t(p.a_ld), w_ld = uint32_t(p.b_ld);
  const uint32_t t_off = (lane >> 3) * t_ld + tk, w_off[2] = {(lane >> 3) * w_ld + wk[0], (lane >> 3) * w_ld + wk[1]};
  // Offsets of a row past the last one are out of range, too: 256 rows of the longest stride do not pass 32 bits.
  const int t_skip = (tw * 16 + nw * 2) * 8, w_skip = nw * 64;
  uint32_t t_bytes, w_bytes;
  int steps;      // of j that there is anything to load for
  const auto set_loads = [&] {
    steps = (j.K + kStep - 1) / kStep;
    t_bytes = j.t_rows * t_ld, w_bytes = j.w_rows * w_ld;
  };
  const auto load_t = [&](int s, int st, int h, int q) {
    load_to_lds<16>(raw_buffer(j.t + int64_t(s) * kStep, t_bytes),
                    lds + st * S::Stage + (tw * 16 + h * 8 + nw * 2 + q) * 1024,
                    tk < j.K - s * kStep ? t_off : kOutOfRange, (t_skip + (h * 8 + q) * 8) * t_ld);
  };
  const auto load_w = [&](int s, int st, int q) {
    const int h = q & 1;
    load_to_lds<16>(raw_buffer(j.w + int64_t(s) * kStep, w_bytes),
                    lds + st * S::Stage + S::TBytes + (nw * 8 + q) * 1024,
                    wk[h] < j.K - s * kStep ? w_off[h] : kOutOfRange, (w_skip + q * 8) * w_ld);
  };
  const auto load_t_scales = [&](int s, int st) {
    // this group's two loads of 64 words, by its first two waves
    const int at = tw * 2 + (nw & 1);
    const int word = at * 64 + lane;
    const bool live = s < steps && nw < 2;
    const uint32_t dst = lds + S::Scales + st * S::ScaleStage + (nw < 2 ? at : S::TS + S::WS) * 256;
    if (MX)     // two loads for each 128 x 4 tile; the next tile of rows lies tile_cols tiles on
      load_to_lds<4>(raw_buffer(j.ts, j.ts_bytes), dst,
                     live ? uint32_t(tw * j.tile_cols + s) * kTileBytes + word % 128 * 4 : kOutOfRange);
    else
      load_to_lds<4>(raw_buffer(j.tf + s * j.tf_ld, uint32_t(j.t_rows) * 4), dst,
                     live ? uint32_t(word) * 4 : kOutOfRange);
  };
  const auto load_w_scales = [&](int s, int st) {
    const int word = nw * 64 + lane;
    const bool live = s < steps && nw < S::WS;
    const uint32_t dst = lds + S::Scales + st * S::ScaleStage + (nw < S::WS ? S::TS + nw : S::TS + S::WS) * 256;
    if (MX)
      load_to_lds<4>(raw_buffer(j.ws, j.ws_bytes), dst,
                     live ? uint32_t(word / 128 * j.tile_cols + s) * kTileBytes + word % 128 * 4 : kOutOfRange);
    else if (DEPTH)
      load_to_lds<4>(raw_buffer(j.wf + s * j.wf_ld, uint32_t(j.w_rows) * 4), dst,
                     live ? uint32_t(word) * 4 : kOutOfRange);
    else        // one word for each 128 outputs
      load_to_lds<4>(raw_buffer(j.wf + s, kAnyBytes), dst,
                     live && word * kTileRows < j.w_rows ? uint32_t(word * ((p.K + kStep - 1) / kStep)) * 4
                                                         : kOutOfRange);
  };

  const uint32_t t_read = (t_first + r) * kStep + ((g ^ (r & 7)) * 16);
  const uint32_t w_read = S::TBytes + (n_first + (r >> 2) * 8 + (r & 3)) * kStep + ((g ^ (r & 7)) * 16);
  const uint32_t ts_read = S::Scales + (MX ? scale_row_offset(t_first + r, 1) : uint32_t(t_first + r) * 4);
  const uint32_t ws_at = S::Scales + S::TS * 256;
  const uint32_t w_lane = n_first + (r >> 2) * 8 + (r & 3);
  const uint32_t ws_read = ws_at + (MX ? scale_row_offset(w_lane, 1) : DEPTH ? w_lane * 4 : n_first / kTileRows * 4);
  v8i w[4], t[4];
  uint32_t ts[MX ? TF : 4], ws[MX || DEPTH ? 4 : 1];
  uint32_t wf[DEPTH && !MX ? 16 : 1];      // block-128 scales of the outputs that the lane has, to multiply with
  const auto read_t = [&](int st, int i) {
    const uint8_t *from = mm_lds + st * S::Stage + i * 16 * kStep;
    t[i & 3] = operand(*reinterpret_cast<const uint4 *>(from + t_read),
                       *reinterpret_cast<const uint4 *>(from + (t_read ^ 64)));
    if (!MX)
      ts[i & 3] = *reinterpret_cast<const uint32_t *>(mm_lds + st * S::ScaleStage + ts_read + i * 64);
  };
  const auto read_w = [&](int st, int n) {
    const uint8_t *from = mm_lds + st * S::Stage + w_row(n) * kStep;
    w[n] = operand(*reinterpret_cast<const uint4 *>(from + w_read),
                   *reinterpret_cast<const uint4 *>(from + (w_read ^ 64)));
  };
  uint4 ts_words[2];
  uint32_t seen;              // block-128 scale that the lane looks at, its row
  const int seen_row = nw < 2 ? t_first + nw * 64 + lane : (tw * 2 + nw - 2) * 64 + lane;
  int first_other;            // step
  const auto read_scales = [&](int st, auto SCALED) {
    const uint8_t *scales = mm_lds + st * S::ScaleStage;
    if (DEPTH && !MX && !SCALED) {
#pragma unroll
      for (int n = 0; n < int(sizeof(wf) / 4); ++n)
        wf[n] = *reinterpret_cast<const uint32_t *>(scales + ws_at + (n_first + g * 8 + n / 8 * 32 + n % 8) * 4);
    } else if (MX) {
      // rows r, r+32, .. of a 128-row block share 16 bytes, rows r+16, .. the ones 256 bytes on
#pragma unroll
      for (int h = 0; h < 2; ++h) ts_words[h] = *reinterpret_cast<const uint4 *>(scales + ts_read + h * 256);
#pragma unroll
      for (int n = 0; n < 4; ++n)
        ws[MX ? n : 0] = *reinterpret_cast<const uint32_t *>(scales + ws_read + (n & 1) * 64 + (n >> 1) * 4);
    } else {
#pragma unroll
      for (int n = 0; n < int(sizeof(ws) / 4); ++n)
        ws[n] = *reinterpret_cast<const uint32_t *>(scales + ws_read + w_row(n) * 4);
      if (kChecked) {
        seen = *reinterpret_cast<const uint32_t *>(scales + (nw < 2 ? S::Scales : ws_at) + seen_row * 4);
        first_other = *other;
      }
    }
  };
  const auto shift_scales = [&] {
    if (MX) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        ts[MX ? h : 0] = ts_words[h].x >> (8 * g), ts[MX ? 2 + h : 0] = ts_words[h].y >> (8 * g);
        ts[MX ? 4 + h : 0] = ts_words[h].z >> (8 * g), ts[MX ? 6 + h : 0] = ts_words[h].w >> (8 * g);
      }
#pragma unroll
      for (int n = 0; n < 4; ++n) ws[MX ? n : 0] >>= 8 * g;
    }
  };
  const auto reads_written = [&] { __builtin_amdgcn_s_waitcnt(0xc07f); };      // lgkmcnt(0)
  const auto reads_done = [&] {
    reads_written();
    shift_scales();
  };
  const auto end_slot = [&] {
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
  };
  // In its slot: without the pins at its end the products move behind the barriers, to where their sums are used.
  const auto pin = [&] {
#pragma unroll
    for (int i = 0; i < TF; ++i)
#pragma unroll
      for (int n = 0; n < 4; ++n) asm volatile("" : "+v"(acc[i][n]));
  };
  const auto multiply_scaled = [&](int st) __attribute__((always_inline)) {
    if (!MX) {
#pragma unroll
      for (int n = 0; n < int(sizeof(ws) / 4); ++n) ws[n] >>= 23;
    }
#pragma unroll
    for (int i = 0; i < TF; ++i) {
      const int s = int(MX ? ts[MX ? i : 0] : ts[i & 3] >> 23);
#pragma unroll
      for (int n = 0; n < 4; ++n) acc[i][n] = mfma(w[n], t[i & 3], acc[i][n], int(ws[MX || DEPTH ? n : 0]), s);
      if (i < 4) read_t(st, i + 4);
      __builtin_amdgcn_sched_barrier(0);
    }
    pin();
  };
  const auto multiply_any = [&](int st) __attribute__((always_inline)) {
    constexpr int kBehind = 4;        // one product, then the sums of the one so many behind: five parts live
    v4f part[kBehind + 1];
    float factor[2];
    const auto add = [&](int at) {                // a block's sums times its scales
      const int i = at / 4, n = at % 4;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        acc[i][n][e] = fmaf(part[at % (kBehind + 1)][e],
                            DEPTH ? factor[i & 1] * __uint_as_float(wf[DEPTH && !MX ? n * 4 + e : 0]) : factor[i & 1],
                            acc[i][n][e]);
    };
#pragma unroll
    for (int i = 0; i < TF; ++i) {
      factor[i & 1] = __uint_as_float(ts[i & 3]) * (DEPTH ? 1.0f : __uint_as_float(ws[0]));
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        const int at = i * 4 + n;
        part[at % (kBehind + 1)] = mfma(w[n], t[i & 3], v4f{0, 0, 0, 0}, kNoScales, kNoScales);
        if (at >= kBehind) add(at - kBehind);
        __builtin_amdgcn_sched_barrier(0);
      }
      if (i < 4) read_t(st, i + 4);
      __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int at = TF * 4 - kBehind; at < TF * 4; ++at) add(at);
    pin();
  };

  // SCALED: the scales go into the products, which takes powers of two. Returns whether the tiles from `block` on
  // have to be done again because there were others.
  const auto run = [&](auto SCALED) __attribute__((always_inline)) {
    set_loads();
    if (tw == 0) {
#pragma unroll
      for (int q = 0; q < 8; ++q) load_w(0, 0, q);
      load_w_scales(0, 0);
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) load_t(0, 0, q >> 1, q & 1);
    load_t_scales(0, 0);
    out = j.out, out_t = j.t_rows, out_w = j.w_rows;
    clear();
    wait_loads<0>();
    reads_written();          // the end offsets
    end_slot();

    // The step after a tile's last is the next tile's first: its loads take the same slots.
    int s = 0, st = 0;        // step to multiply, its stage
    int all = steps;          // of the tile; one of none is a step of zeros
    bool more = true, whole = false;      // whole: all of the stores of the tile before are on the count of loads
    int done = 0;             // steps of all tiles
    uint32_t this_block = block - gridDim.x, last_block = this_block;
    const auto next_step = [&]() __attribute__((always_inline)) {
      int next = s + 1;
      if (next >= all) {
        more = find(ends, j);
        if (!more) j.K = j.t_rows = j.w_rows = 0;
        set_loads();
        next = 0;
      }
      return next;
    };
    // A tile's outputs leave between its last products and the next one's first reads, beside the other group's
    // products: 16 stores a wave, counted as loads are.
    const auto end_step = [&]() __attribute__((always_inline)) {
      whole = false;
      st ^= 1;
      ++done;
      if (++s < all) return true;
      uint8_t *own = mm_lds + kOutputs + wave * 2048;
      whole = out_t == S::TM && out_w == S::TN;
      if (whole)
        store_rows<TF, true>(out, args()->out_ld, out_t, out_w, acc, own, t_first, n_first);
      else
        store_rows<TF, false>(out, args()->out_ld, out_t, out_w, acc, own, t_first, n_first);
      clear();
      out = j.out, out_t = j.t_rows, out_w = j.w_rows;
      last_block = this_block, this_block = block - gridDim.x;
      s = 0, all = steps;
      return more;
    };
    // Loads that may be under way at the end of a slot, the newest ones. lead: the second half's 2, whose use is two
    // slots off, when the rest has to be there; a whole step's 14 when that half has to be. Others: the second half's
    // 2 when the rest of t has to be there; a step's 5 when that half has to be. Stores lie between that half's loads
    // and the step's.
    constexpr int kStores = TF * 2;
    const auto run_group = [&](auto lead) __attribute__((always_inline)) {
      do {
        const int ls = next_step(), to = st ^ 1;
        if (lead) {
#pragma unroll
          for (int n = 0; n < 4; ++n) {
            read_w(st, n);
            load_w(ls, to, n);
          }
          read_scales(st, SCALED);
          load_w(ls, to, 4);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            read_t(st, i);
            if (i < 3)
              load_w(ls, to, 5 + i);
            else
              load_w_scales(ls, to);
          }
          load_t(ls, to, 0, 0);
          load_t(ls, to, 0, 1);
          load_t_scales(ls, to);
          load_t(ls, to, 1, 0);
          load_t(ls, to, 1, 1);
        } else {
#pragma unroll
          for (int n = 0; n < 4; ++n) read_w(st, n);
          load_t(ls, to, 0, 0);
          read_scales(st, SCALED);
          load_t(ls, to, 0, 1);
          read_t(st, 0);
          load_t_scales(ls, to);
          read_t(st, 1);
          load_t(ls, to, 1, 0);
          read_t(st, 2);
          load_t(ls, to, 1, 1);
          read_t(st, 3);
        }
        reads_done();
        if (kChecked && SCALED) {
          // The eight waves look at 64 of a step's scales each, and what one finds ends all waves' next step: by then
          // it is written. (The lead's finds of that next step may be there, too.) 1 .. 254: a power of two in the
          // normal range. Rows past the tile's last have codes 0, and so has a tile of no steps (a group of no tokens),
          // whose scales are zeros that no cast wrote.
          if (__builtin_amdgcn_readfirstlane(first_other) < done) break;
          const bool power =
              __builtin_rotateright32(seen, 23) - 1 < 254 || seen_row >= (nw < 2 ? out_t : out_w) || all == 0;
          if (__ballot(!power) != 0) {
            if (lane == 0) atomicMin(other, done);
            reads_written();
          }
        }
        if (whole)
          wait_loads<(lead ? 14 : 5) + kStores>();
        else
          wait_loads<lead ? 14 : 5>();
        end_slot();
        if (SCALED)
          multiply_scaled(st);
        else
          multiply_any(st);
        wait_loads<2>();
        end_slot();
      } while (end_step());
    };
    if (tw == 0) {
      run_group(std::true_type());
      end_slot();
    } else {
      end_slot();
      run_group(std::false_type());
    }
    wait_loads<0>();          // the out-of-range ones too: nothing is under way into LDS when the workgroup ends
    if (!kChecked || !SCALED || __builtin_amdgcn_readfirstlane(*other) == INT_MAX) return false;
    block = s == 0 ? last_block : this_block;      // the step found is the one before this
    return true;
  };
  if (run(std::integral_constant<bool, MX || kChecked>()) && kChecked) {
    end_slot();
    if (find(p.offs, j)) run(std::false_type());
  }
}

// ------------------------------------------------------------- launch

inline int launch_mm(const void *fn, int64_t grid, int threads, size_t lds, MmParams &p, hipStream_t stream) {
  if (grid > max_grid(threads)) return MX_REARRANGE_ESHAPE;
  void *args[] = {&p};
  const hipError_t e = hipLaunchKernel(fn, dim3(unsigned(grid)), dim3(unsigned(threads)), args, lds, stream);
  return e == hipSuccess ? MX_REARRANGE_OK : MX_REARRANGE_ELAUNCH;
}

// Tiles of TM x TN of the whole product if the rows are spread evenly over the groups (their sizes are on the device).
template <bool DEPTH>
int64_t expected_tiles(const MmParams &p, int TM, int TN) {
  const int64_t groups = DEPTH || p.groups < p.rows ? p.groups : p.rows;
  const int64_t rows = DEPTH ? p.rows : (p.rows + groups - 1) / groups;
  return groups * ((rows + int64_t(TM) - 1) / TM) * ((p.N + TN - 1) / TN);
}

template <bool MX, bool DEPTH, int TF>
int run_stream(MmParams p, hipStream_t stream) {
  p.n_tiles = (p.N + kStreamN - 1) / kStreamN;
  p.m_tiles = (p.rows + TF * 16 - 1) / (TF * 16);
  p.slots = DEPTH ? int64_t(p.groups) * p.m_tiles : row_tiles(p.rows, p.groups, TF * 16);
  return launch_mm(reinterpret_cast<const void *>(&mm_stream_kernel<MX, DEPTH, TF>), p.slots * p.n_tiles,
                   kStreamWaves * kWave, 0, p, stream);
}

template <bool MX, bool DEPTH, int TW, int NW, int TF, int STAGES>
const void *tile_kernel() {
  return reinterpret_cast<const void *>(&mm_tile_kernel<MX, DEPTH, TW, NW, TF, STAGES>);
}

// Launches a tile kernel of shape S (its LDS is more than a launch gets unasked).
template <bool MX, bool DEPTH, class S, bool PAIRED = false>
int run_tiles(MmParams p, const void *fn, hipStream_t stream) {
  constexpr int kMaxDevices = 64;
  static std::once_flag once[kMaxDevices];
  static bool ready[kMaxDevices];
  constexpr int lds = PAIRED ? paired_lds<MX, DEPTH>() : S::Lds;
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxDevices) return MX_REARRANGE_ELAUNCH;
  std::call_once(once[dev], [dev, fn] {
    ready[dev] = hipFuncSetAttribute(fn, hipFuncAttributeMaxDynamicSharedMemorySize, lds) == hipSuccess;
  });
  if (!ready[dev]) return MX_REARRANGE_ELAUNCH;
  p.n_tiles = (p.N + S::TN - 1) / S::TN;
  p.m_tiles = (p.rows + S::TM - 1) / S::TM;
  p.slots = DEPTH ? int64_t(p.groups) * p.m_tiles : row_tiles(p.rows, p.groups, S::TM);
  int64_t grid = slots_for(true, p.slots * p.n_tiles, kDeal);
  if (grid > max_grid(S::WAVES * kWave)) return MX_REARRANGE_ESHAPE;
  // one workgroup per CU that takes tile after tile, where it can look its groups up without memory
  if (PAIRED && p.groups <= kWave && grid > 8 * kDeal) grid = 8 * kDeal;
  return launch_mm(fn, grid, S::WAVES * kWave, lds, p, stream);
}

// Fills in the tiling and launches the kernel that is expected to be fastest, by its time for one step of k: at least
// the latency of a step, and from some number of tiles on a time per tile (the 32 x 128 one also a time for each
// 128 rows of weights from memory, which its tiles of one group share). Measured on one MI355X (us per step; MX and
// block-128, HIP graphs):
//   kernel              latency   per tile            G experts of one size, N, K -> us
//   streamed 16 x 32    0.27      0.8e-3              G 1, 4096, 4096, 16 rows: 9.8 (32 x 128: 15.6, 128 x 128: 23.8)
//   streamed 32 x 32    0.36      1.06e-3             G 1, 4096, 4096, 64 rows: 12.3 (15.6, 24.5)
//   streamed 64 x 32    0.5       1.6e-3              G 1, 8192, 5120, 64 rows: 20.6 (128 x 128: 29.7)
//   tiles 32 x 128      0.5       1.4e-3, 2.6e-3      G 16, 8192, 5120, 16 rows: 120, 5.6 TB/s (128 x 128: 122)
//                                                     G 8, 4096, 7168, 16 rows: 35 (streamed 41, 128 x 128: 62)
//   tiles 128 x 128     1.0       2.6e-3              G 16, 8192, 5120, 64 rows: 144 (32 x 128: 170)
//   paired 256 x 256    1.1       1.6 for each 256    G 16, 8192, 5120, 192 rows: 178 to 190 (128 x 128: 229)
template <bool MX, bool DEPTH>
int run_mm(const MmParams &p, hipStream_t stream) {
  using Few = TileShape<MX, DEPTH, 2, 2, 1, 3>;
  using Small = TileShape<MX, DEPTH, 2, 2, 4, 2>;
  using Paired = TileShape<MX, DEPTH, 2, 4, 8, 2>;
  const auto cost = [&](int TM, int TN, double latency, double per_tile) {
    return fmax(latency, per_tile * double(expected_tiles<DEPTH>(p, TM, TN)));
  };
  const double by[6] = {cost(16, kStreamN, 0.27, 0.8e-3),
                        cost(32, kStreamN, 0.36, 1.06e-3),
                        cost(64, kStreamN, 0.5, 1.6e-3),
                        fmax(cost(Few::TM, Few::TN, 0.5, 1.4e-3), cost(1 << 30, Few::TN, 0.5, 2.6e-3)),
                        cost(Small::TM, Small::TN, 1.0, 2.6e-3),
                        fmax(1.1, 1.6 * double((expected_tiles<DEPTH>(p, Paired::TM, Paired::TN) + 255) / 256))};
  int best = 0;
  for (int i = 1; i < 6; ++i)
    if (by[i] < by[best]) best = i;
  switch (best) {
    case 0: return run_stream<MX, DEPTH, 1>(p, stream);
    case 1: return run_stream<MX, DEPTH, 2>(p, stream);
    case 2: return run_stream<MX, DEPTH, 4>(p, stream);
    case 3: return run_tiles<MX, DEPTH, Few>(p, tile_kernel<MX, DEPTH, 2, 2, 1, 3>(), stream);
    case 4: return run_tiles<MX, DEPTH, Small>(p, tile_kernel<MX, DEPTH, 2, 2, 4, 2>(), stream);
    default: return run_tiles<MX, DEPTH, Paired, true>(p, reinterpret_cast<const void *>(&mm_paired_kernel<MX, DEPTH>),
                                                       stream);
  }
}

// ------------------------------------------------------------- argument checks

constexpr int64_t kMaxDepth = int64_t(1) << 22;    // bytes between rows: 256 rows stay below 2^31
constexpr int64_t kMaxN = (int64_t(1) << 24) - 1;

inline bool aligned16(const void *p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

}  // namespace
