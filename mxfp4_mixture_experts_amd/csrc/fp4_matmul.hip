// Products of two MXFP4 operands, dense or routed to experts, for gfx950:
//
//   out[r, n] = bias[e, n] + sum_k X[src(r), k] * W[e, n, k]
//
// where e is the expert that row r is grouped under (dense: one expert that has
// every row, in order) and src(r) the row of X that it reads.  The codes and the
// scale bytes go to the scaled-FP4 MFMA as they are stored; its sums are fp32.
//
// Few rows are bound by the weights' way from HBM, many by the MFMA: with all CUs
// at it and random codes it runs 32x32x64 at 6.7 PFLOP/s, the clock then at about
// 1.6 GHz.  Two kernels, and three tile shapes, chosen by the rows (launch_out).
#include <type_traits>

#include "kernels.h"
#include "common.h"
#include "fp4_places.h"

namespace mxfp4 {
namespace {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef float f32x2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));

constexpr int kFmtFp4 = 4;  // MFMA operand format code of E2M1
constexpr int kXcds = 8;

__device__ __forceinline__ v8i fp4_operand(u32x4_t v) {
  return v8i{(int)v.x, (int)v.y, (int)v.z, (int)v.w, 0, 0, 0, 0};
}

// The rows [b, f) of expert e in the grouped order, clamped into [0, R].
__device__ __forceinline__ void group_rows(const Fp4MatmulArgs& a, int e, int& b, int& f) {
  if (!a.offsets) {
    b = 0;
    f = a.R;
    return;
  }
  b = min(max(a.offsets[e], 0), a.R);
  f = min(max(a.offsets[e + 1], b), a.R);
}

// The routed row at position p of the grouped order, -1 if there is none.
__device__ __forceinline__ int routed_row(const Fp4MatmulArgs& a, int p, int f) {
  if (p >= f) return -1;
  if (!a.rows) return p;
  const int r = a.rows[p];
  return (unsigned)r < (unsigned)a.R ? r : -1;
}

// Twice the bytes that one column of the product takes in the output.
template <int OUT>
constexpr int kOutBytes2 = OUT == kFp4OutF32 ? 8 : OUT == kFp4OutBf16 ? 4 : 2;

template <int OUT>
__device__ __forceinline__ uint8_t* out_at(const Fp4MatmulArgs& a, int r, int n) {
  return static_cast<uint8_t*>(a.out) + ((size_t)r * a.N + n) * kOutBytes2<OUT> / 2;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2_t{lo, hi}, bf16x2_t));
}

// Eight consecutive outputs of a row (as products, or as four activations), at
// an address that is a multiple of their size (of 16 bytes for fp32).
template <int OUT>
__device__ __forceinline__ void store8(uint8_t* o, const float (&v)[8]) {
  if (OUT == kFp4OutF32) {
    reinterpret_cast<f32x4_t*>(o)[0] = f32x4_t{v[0], v[1], v[2], v[3]};
    reinterpret_cast<f32x4_t*>(o)[1] = f32x4_t{v[4], v[5], v[6], v[7]};
  } else if (OUT == kFp4OutBf16) {
    *reinterpret_cast<u32x4_t*>(o) = u32x4_t{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]),
                                             pack_bf16(v[6], v[7])};
  } else {
    float s[4];
#pragma unroll
    for (int i = 0; i < 4; i++) s[i] = swiglu(v[2 * i], v[2 * i + 1]);
    *reinterpret_cast<uint2*>(o) = make_uint2(pack_bf16(s[0], s[1]), pack_bf16(s[2], s[3]));
  }
}

// Outputs n and n + 1 of row r (those below N), or their activation.
template <int OUT>
__device__ __forceinline__ void store_pair(const Fp4MatmulArgs& a, int r, int n, float v0, float v1) {
  if (n >= a.N) return;
  if (OUT == kFp4OutSwiglu) {
    static_cast<uint16_t*>(a.out)[((size_t)r * a.N + n) / 2] = (uint16_t)f32_to_bf16_any(swiglu(v0, v1));
    return;
  }
  const size_t o = (size_t)r * a.N + n;
  if (OUT == kFp4OutF32) {
    static_cast<float*>(a.out)[o] = v0;
    if (n + 1 < a.N) static_cast<float*>(a.out)[o + 1] = v1;
  } else {
    static_cast<uint16_t*>(a.out)[o] = (uint16_t)f32_to_bf16_any(v0);
    if (n + 1 < a.N) static_cast<uint16_t*>(a.out)[o + 1] = (uint16_t)f32_to_bf16_any(v1);
  }
}

// ---------------------------------------------------------------------------
// few rows
// ---------------------------------------------------------------------------

// A workgroup takes 16 weight rows of one expert and splits K over its four
// waves; 16 routed rows at a time are the MFMA's columns.  Lane l holds weight
// row l % 16 (and routed row l % 16) and block 4 s + l / 16 of K step s.  Bound by
// HBM and, with few experts, by latencies: 4 tokens through 13 experts of 5760 x 2880
// 27.8 us (4.2 TB/s), one token through 4 of them 10.9 (3.2).  The weights are on their
// way before the rows' numbers are back (with the numbers, the inputs and the weights
// one after the other, and the bias at the end, 16 experts took 39.3 us for 31.8).
constexpr int kRowsWaves = 4;
constexpr int kRowsSteps = 6;  // K steps of 128 whose loads are in flight together

template <int OUT>
__global__ __launch_bounds__(kRowsWaves * 64) void fp4_rows_kernel(Fp4MatmulArgs a) {
  __shared__ float part[kRowsWaves][16 * 17];
  __shared__ int rows_lds[16];
  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int c = lane & 15, q = lane >> 4;
  // the blockIdx.y-th expert with rows
  int e = 0;
  if (a.offsets) {
    int left = blockIdx.y;
    e = -1;
    for (int base = 0; base < a.E; base += 64) {
      int b = 0, f = 0;
      if (base + lane < a.E) group_rows(a, base + lane, b, f);
      uint64_t mask = wave_ballot(f > b);
      const int n = __popcll(mask);
      if (left < n) {
        for (int i = 0; i < left; i++) mask &= mask - 1;
        e = base + __builtin_ctzll(mask);
        break;
      }
      left -= n;
    }
    if (e < 0) return;
    e = __builtin_amdgcn_readfirstlane(e);
  }
  int b, f;
  group_rows(a, e, b, f);
  const int KB = a.K >> 5;
  const int steps = (KB + 3) >> 2;
  const int n0 = blockIdx.x * 16;
  const size_t wrow = (size_t)e * a.N + min(n0 + c, a.N - 1);
  const u32x4_t* wq = reinterpret_cast<const u32x4_t*>(a.w) + wrow * KB;
  const uint8_t* wsc = a.ws + wrow * KB;
  // the bias of the end's threads, under way with the weights
  const int nl = 2 * (tid & 7), n = n0 + nl;
  const uint16_t* const bp = a.bias ? a.bias + (size_t)e * a.N : reinterpret_cast<const uint16_t*>(a.w);
  const uint32_t bias0 = bp[a.bias ? min(n, a.N - 1) : 0], bias1 = bp[a.bias ? min(n + 1, a.N - 1) : 0];
  for (int p0 = b; p0 < f; p0 += 16) {
    // the row's number, then the weights, which need none, then the inputs: loads return in order
    const int at = min(p0 + c, f - 1);
    const int listed = *(a.rows ? a.rows + at : reinterpret_cast<const int32_t*>(a.w));  // (not used without a list)
    f32x4_t acc = f32x4_t{0.f, 0.f, 0.f, 0.f};
    for (int s0 = wave; s0 < steps; s0 += kRowsWaves * kRowsSteps) {
      u32x4_t wv[kRowsSteps], xv[kRowsSteps];
      uint32_t wb[kRowsSteps], xb[kRowsSteps];
#pragma unroll
      for (int u = 0; u < kRowsSteps; u++) {
        const int kb = min(4 * (s0 + kRowsWaves * u) + q, KB - 1);  // blocks past K: the last one, masked below
        wv[u] = wq[kb];
        wb[u] = wsc[kb];
      }
      __builtin_amdgcn_sched_barrier(0);
      int named = listed;
      asm volatile("" : "+v"(named));  // (nor is it waited for before the weights are on their way)
      if (!a.rows) named = at;
      const unsigned r = (unsigned)named < (unsigned)a.R ? named : 0u;
      const size_t xrow = a.x_div == 1 ? r : r / (unsigned)a.x_div;
      const u32x4_t* xq = reinterpret_cast<const u32x4_t*>(a.x) + xrow * KB;
      const uint8_t* xsc = a.xs + xrow * KB;
#pragma unroll
      for (int u = 0; u < kRowsSteps; u++) {
        const int kb = min(4 * (s0 + kRowsWaves * u) + q, KB - 1);
        xv[u] = xq[kb];
        xb[u] = xsc[kb];
      }
      __builtin_amdgcn_sched_barrier(0);  // (no load is moved to its use)
#pragma unroll
      for (int u = 0; u < kRowsSteps; u++) {
        // (a block past K has the last one's scales: NaN only where that makes the row NaN too)
        const u32x4_t xm = 4 * (s0 + kRowsWaves * u) + q < KB ? xv[u] : u32x4_t{0, 0, 0, 0};
        acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fp4_operand(wv[u]), fp4_operand(xm), acc, kFmtFp4,
                                                               kFmtFp4, 0, (int)wb[u], 0, (int)xb[u]);
      }
    }
    const int named = a.rows ? listed : at;
    if (tid < 16) rows_lds[tid] = p0 + c < f && (unsigned)named < (unsigned)a.R ? named : -1;
    // lane (c, q): routed row c, weight rows 4 q + i
#pragma unroll
    for (int i = 0; i < 4; i++) part[wave][c * 17 + 4 * q + i] = acc[i];
    __syncthreads();
    // 128 threads: routed row tid / 8, weight rows 2 (tid % 8), + 1
    if (tid < 128) {
      const int row = rows_lds[tid >> 3];
      float v0 = 0.f, v1 = 0.f;
#pragma unroll
      for (int w = 0; w < kRowsWaves; w++) {
        v0 += part[w][(tid >> 3) * 17 + nl];
        v1 += part[w][(tid >> 3) * 17 + nl + 1];
      }
      if (row >= 0 && n < a.N) {
        if (a.bias) {
          uint32_t b0 = bias0, b1 = bias1;
          asm volatile("" : "+v"(b0), "+v"(b1));  // (waited for here)
          v0 += bf16_bits_to_f32(b0);
          v1 += bf16_bits_to_f32(b1);
        }
        store_pair<OUT>(a, row, n, v0, v1);
      }
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------
// tiles
// ---------------------------------------------------------------------------

struct Fp4Tile {
  int e, nt, p0, f;  // expert, weight panel, first position and end of its rows in the grouped order
};

__device__ __forceinline__ int incl_scan(int v, int lane) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int u = __shfl_up(v, d, 64);
    if (lane >= d) v += u;
  }
  return v;
}

// A tile's number within its expert's mt row tiles x NP weight panels: blocks of
// kBlockTiles row tiles, in them panel by panel, so that the 32 tiles that an
// XCD has under way share both their rows and their panels in its L2.
constexpr int kBlockTiles = 8;
__device__ __forceinline__ void place_tile(int local, int mt, int NP, int& m, int& nt) {
  const int block = local / (kBlockTiles * NP);
  const int rest = local - block * kBlockTiles * NP;
  const int height = min(kBlockTiles, mt - block * kBlockTiles);
  nt = rest / height;
  m = block * kBlockTiles + rest - nt * height;
}

// The workgroup's tile: tiles are numbered expert by expert, and every XCD takes
// a contiguous run of the numbers.  False for the surplus workgroups.
template <int TM>
__device__ __forceinline__ bool find_tile(const Fp4MatmulArgs& a, int NP, int lane, Fp4Tile& t) {
  int total = 0;
  if (!a.offsets) {
    total = (a.R + TM - 1) / TM;
  } else {
    for (int base = 0; base < a.E; base += 64) {
      int b = 0, f = 0;
      if (base + lane < a.E) group_rows(a, base + lane, b, f);
      total += __builtin_amdgcn_readlane(incl_scan((f - b + TM - 1) / TM, lane), 63);
    }
  }
  total *= NP;
  const int per = (total + kXcds - 1) / kXcds;
  const int i = blockIdx.x / kXcds;
  const int id = (blockIdx.x % kXcds) * per + i;
  if (i >= per || id >= total) return false;
  if (!a.offsets) {
    int m;
    place_tile(id, total / NP, NP, m, t.nt);
    t.e = 0;
    t.p0 = m * TM;
    t.f = a.R;
    return true;
  }
  int before = 0;
  for (int base = 0; base < a.E; base += 64) {
    int b = 0, f = 0;
    if (base + lane < a.E) group_rows(a, base + lane, b, f);
    const int cnt = (f - b + TM - 1) / TM * NP;
    const int incl = incl_scan(cnt, lane) + before;
    const uint64_t hit = wave_ballot(id >= incl - cnt && id < incl);
    if (hit) {
      const int src = __builtin_ctzll(hit);
      const int local = id - __builtin_amdgcn_readlane(incl - cnt, src);
      t.e = base + src;
      b = __builtin_amdgcn_readlane(b, src);
      t.f = __builtin_amdgcn_readlane(f, src);
      int m;
      place_tile(local, (t.f - b + TM - 1) / TM, NP, m, t.nt);
      t.p0 = b + m * TM;
      return true;
    }
    before = __builtin_amdgcn_readlane(incl, 63);
  }
  return false;
}

// Keeps the compiler's scheduler from moving instructions across.
__device__ __forceinline__ void pipeline_fence() { __builtin_amdgcn_sched_barrier(0); }

// Every wave's LDS reads and writes before it are done behind it; loads from
// memory stay under way.
__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// 16 bytes a lane from memory into LDS: lane l's go to the wave's destination +
// 16 l.  In asm, because the compiler waits for the arrival of every such load
// before any LDS read that it cannot tell apart from the destination; here
// the arrival is waited for with vmcnt before the barrier behind which the
// data are read.  (No output registers; the nop is the wait state between the
// write of m0 and its use.  The compiler keeps no value in m0, a reserved register that
// a clobber list may not name; nothing else here uses it.)
__device__ __forceinline__ void dma16(const void* src, uint32_t lds_off) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(lds_off), "v"(src)
               : "memory");
}

// Waits until at most N of the wave's loads are under way.
template <int N>
__device__ __forceinline__ void wait_loads() {
  static_assert(N < 64, "six bits");
  __builtin_amdgcn_s_waitcnt(0x0f70 | (N & 15) | (N >> 4) << 14);
  asm volatile("" ::: "memory");
}

// K step j of a stage is the blocks first_block(j) and first_block(j) + 2.
__device__ __forceinline__ constexpr int first_block(int j) { return (j & 2) * 2 + (j & 1); }

// The order of a row's eight blocks of a stage in LDS, in which the lanes that
// read one block of different rows meet different banks.
__device__ __forceinline__ int row_swizzle(int r) { return (r & 7) ^ ((r >> 3) & 1); }

// Four waves side by side along the weight rows.  The weights are the MFMA's
// operand A, the activations operand B: a lane of an accumulator then holds
// one routed row and runs of four consecutive outputs.  Every wave multiplies
// all the tile's routed rows, so a tile with few of them leaves whole
// sub-tiles out.
//
// K goes by stages of eight blocks (256 elements): a row's 128 bytes of codes.  A
// weight row belongs to one wave, so its codes go straight to registers, a stage
// and a half ahead, by loads of 16 rows x 64 bytes, which a CU takes from L2 at 149
// bytes a ns (32 rows x 32 bytes: 72); an exchange between the lanes makes the
// MFMA's operands of them.  The activations, which all waves share, go straight to
// two slots of LDS.  A row's scale bytes start anywhere: a window of 32 blocks comes
// as the three aligned 16-byte pieces that hold it (none without a byte of the row);
// a thread a row shifts them into place and splits them into a word a stage and
// half wave, of which the MFMA picks a byte.
//
// Two workgroups share a CU, two waves a SIMD: one wave a SIMD with half as many
// accumulators again came to 0.6 of the rate, its loads, waits, first and last
// steps in line with its products.  Loads are spread between the products, one
// behind every second: a load holds up the products of a lone wave for 32 cycles,
// those of two for 15.  4096 x 5760 x 2880 runs at 2.4 PFLOP/s with its operands in the
// last-level cache and at 2.0 from HBM (736 tiles on 512 places), 8192^3 at 3.0 and 2.8.
template <int MT, int NT>
struct TileShape {
  static constexpr int kWaves = 4, kThreads = kWaves * 64;
  static constexpr int TM = MT * 32, TN = kWaves * NT * 32, kRows = TM + TN;
  static constexpr int kSlot = TM * 128;  // a stage of activations
  static constexpr int kScalePieces = kRows * 3 / 64;  // 1 KB pieces of a window of scale bytes
  static constexpr int kRawAt = 2 * kSlot;             // a window as it comes
  static constexpr int kScalesAt = kRawAt + kRows * 48;  // eight stages' words: [stage][row][half]
  static constexpr int kBiasAt = kScalesAt + 8 * kRows * 8;
  static constexpr int kRowsAt = kBiasAt + TN * 4;
  static constexpr int kSrcAt = kRowsAt + TM * 4;
  static constexpr int kLds = kSrcAt + TM * 4;
  static_assert(kRows * 3 % 64 == 0, "whole pieces");
  static_assert(kLds <= 80 * 1024, "half the LDS of a CU");
};

template <int MT, int NT, int OUT>
__global__ __launch_bounds__(256, 2) void fp4_tile_kernel(Fp4MatmulArgs a, int vec) {
  using S = TileShape<MT, NT>;
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  float* const bias_lds = reinterpret_cast<float*>(lds + S::kBiasAt);
  int* const rows_lds = reinterpret_cast<int*>(lds + S::kRowsAt);  // the tile's routed rows, -1 if none
  int* const src_lds = reinterpret_cast<int*>(lds + S::kSrcAt);    // X's rows that they read
  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l32 = lane & 31, half = lane >> 5;
  Fp4Tile t;
  if (!find_tile<S::TM>(a, (a.N + S::TN - 1) / S::TN, lane, t)) return;
  const int KB = a.K >> 5;
  const int last = (KB - 1) >> 3;  // the last stage
  const int n0 = t.nt * S::TN;

  // this wave's weight rows
  const int wn0 = fp4_wave_first(n0 + wave * NT * 32, a.N);
  const int wrows = fp4_wave_rows(n0 + wave * NT * 32, a.N, NT * 32);
  const __amdgpu_buffer_rsrc_t wsrc = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint8_t*>(a.w + ((size_t)t.e * a.N + wn0) * KB * 16), (short)0, wrows * KB * 16, 0x00020000);
  int woff[NT][2];
#pragma unroll
  for (int n = 0; n < NT; n++)
#pragma unroll
    for (int u = 0; u < 2; u++) woff[n][u] = fp4_row_at(n, u, lane, wrows, KB);
  u32x4_t w[2][NT][4];
  // piece i of a stage's 4 NT: sub-tile i / 4, blocks 4 (i / 2 % 2) .. + 3, rows 16 (i % 2) .. + 15.
  // Every lane's offset lies in the wave's rows: a buffer's bounds are not checked against
  // an offset in a scalar register, so none is left to them.
  auto load_w = [&](int s, int i) {
    return __builtin_amdgcn_raw_buffer_load_b128(wsrc, woff[i >> 2][i & 1] + fp4_block_at(s, i >> 1 & 1, lane, KB), 0,
                                                 0);
  };
  // the rows and the bias first: the barrier waits for them, not for the weights
  static_assert(S::TM <= S::kThreads, "a row a thread");
  const int row0 = tid < S::TM ? routed_row(a, t.p0 + tid, t.f) : -1;
  uint32_t bias0[(S::TN + S::kThreads - 1) / S::kThreads];
#pragma unroll
  for (int i = 0; i * S::kThreads < S::TN; i++)
    bias0[i] = a.bias ? a.bias[(size_t)t.e * a.N + min(n0 + tid + i * S::kThreads, a.N - 1)] : 0;
  pipeline_fence();
#pragma unroll
  for (int i = 0; i < 4 * NT; i++) w[0][i >> 2][i & 3] = load_w(0, i);
  pipeline_fence();
  if (tid < S::TM) {
    rows_lds[tid] = row0;
    // rows past the end read a valid one, whose products are not stored
    src_lds[tid] = row0 < 0 ? 0 : a.x_div == 1 ? row0 : row0 / a.x_div;
  }
#pragma unroll
  for (int i = 0; i * S::kThreads < S::TN; i++)
    if (tid + i * S::kThreads < S::TN) bias_lds[tid + i * S::kThreads] = bf16_bits_to_f32(bias0[i]);
  lds_barrier();

  // activations: a wave brings MT pieces of 8 rows; lane l brings row l / 8's LDS
  // place l % 8, the block place ^ row_swizzle(row)
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)lds;
  const int xblk = (lane & 7) ^ (lane >> 3) ^ (wave & 1);
  const int* const x_src = src_lds + 8 * wave + (lane >> 3);
  auto x_piece = [&](int s, int slot, int p) {
    const int off = min(8 * s + xblk, KB - 1) * 16;  // blocks past K: the last one, masked later
    dma16(a.x + (size_t)(uint32_t)x_src[32 * p] * (uint32_t)(KB * 16) + off,
          lds0 + slot * S::kSlot + (wave + S::kWaves * p) * 1024);
  };
  auto bring_x = [&](int s, int slot) {
#pragma unroll
    for (int p = 0; p < MT; p++) x_piece(min(s, last), slot, p);
  };
  bring_x(0, 0);

  // scales: tile row i is X's (i < TM), then W's row n0 + i - TM.  Piece c of the
  // window's kRows x 3 goes to its place in order; a piece past the row's last
  // byte reads the one with that byte again.
  auto scale_row = [&](int i) -> uintptr_t {
    return i < S::TM ? reinterpret_cast<uintptr_t>(a.xs) + (size_t)(uint32_t)src_lds[i] * (uint32_t)KB
                     : reinterpret_cast<uintptr_t>(a.ws + (size_t)t.e * a.N * KB) +
                           (size_t)(uint32_t)min(n0 + i - S::TM, a.N - 1) * (uint32_t)KB;
  };
  auto bring_scales = [&](int v) {
#pragma unroll 1
    for (int p = wave; p < S::kScalePieces; p += S::kWaves) {
      const int c = 64 * p + lane;
      const int i = c / 3;
      const uintptr_t row = scale_row(i);
      const uintptr_t at = min((row & ~(uintptr_t)15) + 32 * v + 16 * (c - 3 * i), (row + KB - 1) & ~(uintptr_t)15);
      dma16(reinterpret_cast<const void*>(at), lds0 + S::kRawAt + p * 1024);
    }
  };
  bring_scales(0);
  auto put_scales = [&](int v) {
#pragma unroll 1
    for (int i = tid; i < S::kRows; i += S::kThreads) {
      const int shift = (int)(scale_row(i) & 15);
      const uint32_t* q = reinterpret_cast<const uint32_t*>(lds + S::kRawAt + i * 48 + (shift & ~3));
      uint32_t r[9], d[8];
#pragma unroll
      for (int j = 0; j < 9; j++) r[j] = q[j];
#pragma unroll
      for (int j = 0; j < 8; j++) d[j] = __builtin_amdgcn_alignbyte(r[j + 1], r[j], shift & 3);
#pragma unroll
      for (int j = 0; j < 4; j++)
        *reinterpret_cast<uint2*>(lds + S::kScalesAt + ((4 * (v & 1) + j) * S::kRows + i) * 8) =
            make_uint2(__builtin_amdgcn_perm(d[2 * j + 1], d[2 * j], 0x05040100u),
                       __builtin_amdgcn_perm(d[2 * j + 1], d[2 * j], 0x07060302u));
    }
  };

  const int xoff = l32 * 128 + ((2 * half ^ row_swizzle(l32)) << 4);  // block 2 half; K step j: ^ its first block << 4

  // The tile with its first MA sub-tiles of routed rows.
  auto run = [&](auto mac) {
    constexpr int MA = decltype(mac)::value;
    // Lane (l32, half) holds routed row l32 of each 32 x 32 block and outputs
    // 8 g + 4 half + i of it in element 4 g + i; the sums start at the bias.
    v16f acc[NT][MA];
#pragma unroll
    for (int n = 0; n < NT; n++)
#pragma unroll
      for (int g = 0; g < 4; g++) {
        const f32x4_t v = *reinterpret_cast<const f32x4_t*>(bias_lds + (wave * NT + n) * 32 + 8 * g + 4 * half);
#pragma unroll
        for (int m = 0; m < MA; m++)
#pragma unroll
          for (int i = 0; i < 4; i++) acc[n][m][4 * g + i] = v[i];
      }
    u32x4_t x[MA];  // a K step's activations
    struct Scales {
      int w[NT], x[MA];
    };
    auto read_x = [&](int slot, int j, int m) {
      x[m] = *reinterpret_cast<const u32x4_t*>(lds + slot * S::kSlot + (xoff ^ first_block(j) << 4) + m * 4096);
    };
    auto read_scales = [&](Scales& c, int s) {
      const uint8_t* q = lds + S::kScalesAt + (s & 7) * (S::kRows * 8) + l32 * 8 + half * 4;
#pragma unroll
      for (int n = 0; n < NT; n++) c.w[n] = *reinterpret_cast<const int*>(q + (S::TM + (wave * NT + n) * 32) * 8);
#pragma unroll
      for (int m = 0; m < MA; m++) c.x[m] = *reinterpret_cast<const int*>(q + m * 256);
    };
    // the pieces of sub-tile n, blocks 4 v .. + 3, become the operands of K steps 2 v and 2 v + 1
    auto exchange = [&](int set, int n, int v) {
#pragma unroll
      for (int i = 0; i < 4; i++) {
        const auto p = __builtin_amdgcn_permlane16_swap(w[set][n][2 * v][i], w[set][n][2 * v + 1][i], false, false);
        w[set][n][2 * v][i] = p[0];
        w[set][n][2 * v + 1][i] = p[1];
      }
    };
    Scales sc;
    auto multiply = [&](int set, int n, int m, auto jc) {
      constexpr int J = decltype(jc)::value;
      acc[n][m] =
          __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fp4_operand(w[set][n][J]), fp4_operand(x[m]), acc[n][m],
                                                          kFmtFp4, kFmtFp4, J, sc.w[n], J, sc.x[m]);
    };
    using J0 = std::integral_constant<int, 0>;
    using J1 = std::integral_constant<int, 1>;
    using J2 = std::integral_constant<int, 2>;
    using J3 = std::integral_constant<int, 3>;

    wait_loads<0>();  // the first stage's activations and window of scales
    lds_barrier();
    bring_x(1, 1);
#pragma unroll
    for (int i = 0; i < 4 * NT; i++)
      if ((i & 2) == 0) w[1][i >> 2][i & 3] = load_w(1, i);
    put_scales(0);
    lds_barrier();
    read_scales(sc, 0);
#pragma unroll
    for (int m = 0; m < MA; m++) read_x(0, 0, m);
    // scale bytes of the last stage's blocks that exist
    const int left = KB - 8 * last;
    uint32_t kept = 0;
#pragma unroll
    for (int j = 0; j < 4; j++) kept |= first_block(j) + 2 * half < left ? 0xffu << 8 * j : 0u;
    auto keep_scales = [&](uint32_t mask) {
#pragma unroll
      for (int n = 0; n < NT; n++) sc.w[n] &= (int)mask;
#pragma unroll
      for (int m = 0; m < MA; m++) sc.x[m] &= (int)mask;
    };
    // Stage s, s % 2 = set.  Each K step goes over the wave's weight sub-tiles;
    // behind the last one's product with a sub-tile of activations its registers
    // take the next K step's.  The weights of the second half of stage s + 1 are
    // asked for during the first half, those of the first half of stage s + 2
    // during the second, into the registers that the half stage before set free.
    // Before the last sub-tile of the last K step every wave has read the stage's
    // slot, which then takes the activations of stage s + 2.
    auto stage = [&](int s, auto setc) {
      constexpr int set = decltype(setc)::value;
      // The next window of scales: asked for at its predecessor's first stage, here
      // with that stage's barrier, put in place in the third, read in the fourth.
      if (set == 0 && s / 4 < (KB - 1) >> 5) {
        if ((s & 3) == 0) bring_scales(s / 4 + 1);
        else put_scales(s / 4 + 1);
      }
      Scales next;
      exchange(set, 0, 0);
      pipeline_fence();
      auto step = [&](auto jc) {
        constexpr int J = decltype(jc)::value;
#pragma unroll
        for (int n = 0; n < NT; n++) {
          if (J == 3 && n == NT - 1) {
            // the next stage's activations were asked for behind the last barrier;
            // 4 NT - 1 loads of weights followed
            wait_loads<4 * NT - 2>();
            lds_barrier();
            read_scales(next, s + 1);
            pipeline_fence();
          }
#pragma unroll
          for (int m = 0; m < MA; m++) {
            multiply(set, n, m, jc);
            if (n == NT - 1) read_x(J < 3 ? set : 1 - set, (J + 1) & 3, m);
            if (J == 0 && m == 0 && n + 1 < NT) exchange(set, n + 1, 0);
            if (J == 1 && m == 0) exchange(set, n, 1);
            if (m == MA / 2) {
              if (J < 2) w[1 - set][n][2 + (J & 1)] = load_w(s + 1, 4 * n + 2 + (J & 1));
              else w[set][n][J & 1] = load_w(s + 2, 4 * n + (J & 1));
            }
            if (J == 3 && n == NT - 1) {
#pragma unroll
              for (int i = m * MT / MA; i < (m + 1) * MT / MA; i++) x_piece(min(s + 2, last), set, i);
            }
            pipeline_fence();
          }
        }
      };
      step(J0{});
      step(J1{});
      step(J2{});
      step(J3{});
      sc = next;
    };
    // Stages in pairs.  A last one with an odd number goes with them, its blocks past
    // K (the last one's codes again) under scale byte 0 on both sides: products below
    // 2^-240, that change no sum.  A last one with an even
    // number follows, with the K steps that it has.
    for (int s = 0; s < last; s += 2) {
      stage(s, J0{});
      keep_scales(s + 1 == last ? kept : ~0u);  // (no branch: with one the accumulators were spilled)
      stage(s + 1, J1{});
    }
    keep_scales(kept);
    const int rest = last & 1 ? 0 : left;
    auto tail = [&](auto jc) {
      constexpr int J = decltype(jc)::value;
      if (first_block(J) >= rest) return;
#pragma unroll
      for (int n = 0; n < NT; n++) {
        if ((J & 1) == 0) exchange(0, n, J >> 1);
#pragma unroll
        for (int m = 0; m < MA; m++) {
          if (J > 0 && n == 0) read_x(0, J, m);
          multiply(0, n, m, jc);
        }
      }
    };
    tail(J0{});
    tail(J1{});
    tail(J2{});
    tail(J3{});
    wait_loads<0>();  // nothing comes into LDS any more

    // Exchanged between the half waves, the lower one has the eight outputs
    // 8 g .. + 7 of its row for even g, the upper one for odd g.
    const int nw = n0 + wave * NT * 32;
    auto eight = [&](int n, int m, int g, float(&v)[8]) {
#pragma unroll
      for (int i = 0; i < 4; i++) {
        const auto p = __builtin_amdgcn_permlane32_swap(__float_as_uint(acc[n][m][4 * g + i]),
                                                        __float_as_uint(acc[n][m][4 * g + 4 + i]), false, false);
        v[i] = __uint_as_float(p[0]);
        v[4 + i] = __uint_as_float(p[1]);
      }
    };
    if (vec && nw + NT * 32 <= a.N) {
#pragma unroll
      for (int m = 0; m < MA; m++) {
        const int r = rows_lds[32 * m + l32];
        uint8_t* o = out_at<OUT>(a, max(r, 0), nw + 8 * half);
#pragma unroll
        for (int n = 0; n < NT; n++)
#pragma unroll
          for (int g = 0; g < 4; g += 2) {
            float v[8];
            eight(n, m, g, v);
            if (r >= 0) store8<OUT>(o + (32 * n + 8 * g) * kOutBytes2<OUT> / 2, v);
          }
      }
      return;
    }
#pragma unroll
    for (int m = 0; m < MA; m++) {
      const int r = rows_lds[32 * m + l32];
#pragma unroll
      for (int n = 0; n < NT; n++)
#pragma unroll
        for (int g = 0; g < 4; g += 2) {
          float v[8];
          eight(n, m, g, v);
          if (r >= 0) {
#pragma unroll
            for (int i = 0; i < 8; i += 2) store_pair<OUT>(a, r, nw + 32 * n + 8 * (g + half) + i, v[i], v[i + 1]);
          }
        }
    }
  };
  const int subs = (min(t.f - t.p0, S::TM) + 31) >> 5;
  if (MT >= 4 && subs >= 4) run(std::integral_constant<int, MT >= 4 ? 4 : 1>{});
  else if (MT >= 3 && subs == 3) run(std::integral_constant<int, MT >= 3 ? 3 : 1>{});
  else if (MT >= 2 && subs >= 2) run(std::integral_constant<int, MT >= 2 ? 2 : 1>{});
  else run(std::integral_constant<int, 1>{});
}

// At most so many tiles: R / TM whole row tiles and one broken one for each expert
// with rows.
template <int MT, int NT>
long long tiles(const Fp4MatmulArgs& a) {
  using S = TileShape<MT, NT>;
  const long long mt = a.offsets ? a.R / S::TM + (long long)min(a.E, a.R) : ((long long)a.R + S::TM - 1) / S::TM;
  return mt * ((a.N + S::TN - 1) / S::TN);
}

template <int MT, int NT, int OUT>
hipError_t launch_tiles(const Fp4MatmulArgs& a, hipStream_t stream) {
  using S = TileShape<MT, NT>;
  static DynLdsLimit limit(reinterpret_cast<const void*>(fp4_tile_kernel<MT, NT, OUT>), S::kLds);
  const hipError_t e = limit.ensure();
  if (e != hipSuccess) return e;
  const long long grid = (tiles<MT, NT>(a) + kXcds - 1) / kXcds * kXcds;
  const int vec = a.N % 8 == 0 && (reinterpret_cast<uintptr_t>(a.out) & 15u) == 0;
  hipLaunchKernelGGL((fp4_tile_kernel<MT, NT, OUT>), dim3((unsigned)grid), dim3(S::kThreads), S::kLds, stream, a, vec);
  return hipGetLastError();
}

template <int OUT>
hipError_t launch_rows(const Fp4MatmulArgs& a, hipStream_t stream) {
  const unsigned ne = a.offsets ? (unsigned)min(a.E, a.R) : 1u;
  hipLaunchKernelGGL(fp4_rows_kernel<OUT>, dim3((unsigned)((a.N + 15) / 16), ne), dim3(kRowsWaves * 64), 0, stream, a);
  return hipGetLastError();
}

// Few rows an expert: 16 x 16 blocks that stream the weights, against the smallest tiles (us, two
// or three sets of operands in turn).  A workgroup of either pays a chain of latencies, and there
// are many more of the blocks': they win while they are few (1 x 5760 x 2880 4.6 against 8.5, 16 rows
// 5.7 / 10.3, from HBM 5.8 / 13.6; 16 routed rows over 32 experts of 1024 x 2304 7.9 / 11.4), and
// beyond that where the rows are long and do not start line by line in the same place (16 routed
// rows of 5760 x 2880 23.6 / 26.7, 64 of them 62 / 65, 64 over 64 experts of 2880 x 2880 44 / 49); else
// the tiles do (16 routed rows of 5760 x 1024 34 / 14, of 5760 x 4096 72 / 44, 1 x 40000 x 2048 19 / 14).
// A block goes over its expert's rows by sixteens, and a token's experts differ, so up to 32 tokens
// are two rounds: all 32 on the same 2 of 128 experts of 2880 x 2880 11.8 / 10.6, on the same 8
// 20.8 / 13.6; 128 tokens on the same 8 of 512 experts of 1024 x 1024 would take 87 / 18.
bool takes_rows(const Fp4MatmulArgs& a, long long groups) {
  const long long blocks = groups * ((a.N + 15) / 16);
  const bool few = blocks <= (a.K > 1024 ? 1024 : 512), long_rows = a.K >= 2560 && a.K % 256 != 0;
  return (few || long_rows) && (a.offsets ? a.R <= 2 * groups && a.T <= 32 : a.R <= 16);
}

template <int OUT>
hipError_t launch_out(const Fp4MatmulArgs& a, hipStream_t stream) {
  const long long groups = a.offsets ? min(a.E, a.R) : 1;
  if (takes_rows(a, groups)) return launch_rows<OUT>(a, stream);
  // The smallest tiles that give no CU two workgroups, for a tile's time hardly depends on how
  // many run (17 to 256 rows of 5760 x 2880: 64 x 128 tiles 10.0 to 12.4 us, 128 x 128 11.6 to 14.7,
  // 128 x 256 14.8 to 19.2; 1024 rows: 24.2, 21.9, 21.0); and the smallest where an expert has few
  // rows (1024 routed rows over 32 experts of 5760 x 2880: 88 us in 64 x 128 tiles, 93 in 128 x 256,
  // their numbers falling as a power of the expert's 97 and 104; 2048 rows 122 and 97, 126 and 112).
  // Of 156 sizes with all three timed it misses the best by more than 8 percent at 7, by a third at
  // most (512 rows over 8 experts of 2880 x 2880 21.8 us, 16.5 in the smallest: its count of tiles
  // takes a broken one for every expert).
  constexpr long long kCus = 256;
  if (tiles<2, 1>(a) <= kCus || (a.offsets && a.R <= 32 * groups)) return launch_tiles<2, 1, OUT>(a, stream);
  if (tiles<4, 1>(a) <= kCus) return launch_tiles<4, 1, OUT>(a, stream);
  return launch_tiles<4, 2, OUT>(a, stream);
}

}  // namespace

hipError_t launch_fp4_matmul(const Fp4MatmulArgs& a, int out_kind, hipStream_t stream) {
  switch (out_kind) {
    case kFp4OutF32: return launch_out<kFp4OutF32>(a, stream);
    case kFp4OutBf16: return launch_out<kFp4OutBf16>(a, stream);
    default: return launch_out<kFp4OutSwiglu>(a, stream);
  }
}

}  // namespace mxfp4
