// Products of two MXFP4 operands, dense or routed to experts, for gfx950:
//
//   out[r, n] = bias[e, n] + sum_k X[src(r), k] * W[e, n, k]
//
// where e is the expert that row r is grouped under (dense: one expert that has
// every row, in order) and src(r) the row of X that it reads.
#include <type_traits>

#include "kernels.h"
#include "common.h"

namespace mxfp4 {
namespace {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v16f __attribute__((ext_vector_type(16)));

constexpr int kFmtFp4 = 4;  // MFMA operand format code of E2M1
constexpr int kXcds = 8;

// 16 bytes a lane from global memory into LDS: lane l's go to the wave's
// destination + 16 l.  In asm, because the compiler waits for such a load's
// arrival before any LDS read that it cannot tell apart from the destination;
// here every arrival is waited for with s_waitcnt vmcnt before the barrier
// behind which the data are read.  (No output registers; the nop is the wait
// state between the write of m0 and its use.  Nothing else here uses m0.)
__device__ __forceinline__ void dma16(const void* src, uint32_t lds_off) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(lds_off), "v"(src)
               : "memory");
}

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

// V consecutive outputs of row r from column n on (V = 8: all of them exist and
// the row's start and n allow 16-byte stores of fp32, of bf16, or 8-byte
// stores of activations; V = 2: n + 1 may be past N).
template <int OUT>
__device__ __forceinline__ void store8(const Fp4MatmulArgs& a, int r, int n, const float (&v)[8]) {
  if (OUT == kFp4OutF32) {
    f32x4_t* o = reinterpret_cast<f32x4_t*>(static_cast<float*>(a.out) + (size_t)r * a.N + n);
    o[0] = f32x4_t{v[0], v[1], v[2], v[3]};
    o[1] = f32x4_t{v[4], v[5], v[6], v[7]};
  } else if (OUT == kFp4OutBf16) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; i++) w[i] = f32_to_bf16_any(v[2 * i]) | f32_to_bf16_any(v[2 * i + 1]) << 16;
    *reinterpret_cast<u32x4_t*>(static_cast<uint16_t*>(a.out) + (size_t)r * a.N + n) = u32x4_t{w[0], w[1], w[2], w[3]};
  } else {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; i++) w[i] = f32_to_bf16_any(swiglu(v[2 * i], v[2 * i + 1]));
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + ((size_t)r * a.N + n) / 2) =
        make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
  }
}

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
// row l % 16 (and routed row l % 16) and block 4 s + l / 16 of K step s.
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
  for (int p0 = b; p0 < f; p0 += 16) {
    const int r = routed_row(a, p0 + c, f);
    const size_t xrow = r < 0 ? 0 : a.x_div == 1 ? r : r / a.x_div;
    const u32x4_t* xq = reinterpret_cast<const u32x4_t*>(a.x) + xrow * KB;
    const uint8_t* xsc = a.xs + xrow * KB;
    if (tid < 16) rows_lds[tid] = r;
    f32x4_t acc = f32x4_t{0.f, 0.f, 0.f, 0.f};
    for (int s0 = wave; s0 < steps; s0 += kRowsWaves * kRowsSteps) {
      u32x4_t wv[kRowsSteps], xv[kRowsSteps];
      uint32_t wb[kRowsSteps], xb[kRowsSteps];
#pragma unroll
      for (int u = 0; u < kRowsSteps; u++) {
        const int kb = min(4 * (s0 + kRowsWaves * u) + q, KB - 1);  // blocks past K: the last one, masked below
        wv[u] = wq[kb];
        wb[u] = wsc[kb];
        xv[u] = xq[kb];
        xb[u] = xsc[kb];
      }
#pragma unroll
      for (int u = 0; u < kRowsSteps; u++) {
        const int s = s0 + kRowsWaves * u;
        if (s < steps) {
          const u32x4_t xm = 4 * s + q < KB ? xv[u] : u32x4_t{0, 0, 0, 0};
          acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fp4_operand(wv[u]), fp4_operand(xm), acc, kFmtFp4,
                                                                 kFmtFp4, 0, (int)wb[u], 0, (int)xb[u]);
        }
      }
    }
    // lane (c, q): routed row c, weight rows 4 q + i
#pragma unroll
    for (int i = 0; i < 4; i++) part[wave][c * 17 + 4 * q + i] = acc[i];
    __syncthreads();
    // 128 threads: routed row tid / 8, weight rows 2 (tid % 8), + 1
    if (tid < 128) {
      const int row = rows_lds[tid >> 3];
      const int nl = 2 * (tid & 7), n = n0 + nl;
      float v0 = 0.f, v1 = 0.f;
#pragma unroll
      for (int w = 0; w < kRowsWaves; w++) {
        v0 += part[w][(tid >> 3) * 17 + nl];
        v1 += part[w][(tid >> 3) * 17 + nl + 1];
      }
      if (row >= 0 && n < a.N) {
        if (a.bias) {
          const uint16_t* bp = a.bias + (size_t)e * a.N;
          v0 += bf16_bits_to_f32(bp[n]);
          v1 += bf16_bits_to_f32(bp[min(n + 1, a.N - 1)]);
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

// The workgroup's tile: tiles are numbered expert by expert, weight panel by
// weight panel, the panel's row tiles next to each other, and every XCD takes
// a contiguous run of the numbers.  False for the surplus workgroups.
template <int TM>
__device__ __forceinline__ bool find_tile(const Fp4MatmulArgs& a, int NT, int lane, Fp4Tile& t) {
  int total = 0;
  for (int base = 0; base < a.E; base += 64) {
    int b = 0, f = 0;
    if (base + lane < a.E) group_rows(a, base + lane, b, f);
    int v = (f - b + TM - 1) / TM;
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) v += __shfl_xor(v, d, 64);
    total += v;
  }
  total *= NT;
  const int per = (total + kXcds - 1) / kXcds;
  const int i = blockIdx.x / kXcds;
  const int id = (blockIdx.x % kXcds) * per + i;
  if (i >= per || id >= total) return false;
  int before = 0;
  for (int base = 0; base < a.E; base += 64) {
    int b = 0, f = 0;
    if (base + lane < a.E) group_rows(a, base + lane, b, f);
    const int cnt = (f - b + TM - 1) / TM * NT;
    const int incl = incl_scan(cnt, lane) + before;
    const uint64_t hit = wave_ballot(id >= incl - cnt && id < incl);
    if (hit) {
      const int src = __builtin_ctzll(hit);
      const int local = id - __shfl(incl - cnt, src, 64);
      b = __shfl(b, src, 64);
      f = __shfl(f, src, 64);
      const int mt = (f - b + TM - 1) / TM;
      t.e = __builtin_amdgcn_readfirstlane(base + src);
      t.nt = __builtin_amdgcn_readfirstlane(local / mt);
      t.p0 = __builtin_amdgcn_readfirstlane(b + local % mt * TM);
      t.f = __builtin_amdgcn_readfirstlane(f);
      return true;
    }
    before = __shfl(incl, 63, 64);
  }
  return false;
}

// Keeps the compiler's scheduler from moving instructions across.
__device__ __forceinline__ void pipeline_fence() { __builtin_amdgcn_sched_barrier(0); }

// Waits until at most N of the wave's loads are under way.
template <int N>
__device__ __forceinline__ void wait_loads() {
  static_assert(N < 64, "six bits");
  __builtin_amdgcn_s_waitcnt(0x0f70 | (N & 15) | (N >> 4) << 14);
}

// The products of X rows (MFMA operand B) and W rows (operand A): a lane of an
// accumulator then holds one routed row and runs of four consecutive outputs.
// Four waves side by side along the weight rows; every wave multiplies all the
// tile's routed rows, so a tile with few of them leaves whole sub-tiles out.
//
// K goes by stages of four blocks (128 elements).  A ring of four stages in
// LDS, 64 bytes a row, filled by direct loads; a row's blocks lie in an order
// (block ^ row / 2) in which eight lanes that read one block of eight rows meet
// distinct banks.  Scale bytes come in groups of 16 blocks: a row's bytes start
// anywhere, so two aligned 16-byte pieces hold them (clamped to the piece with
// the row's last byte), which one thread a row shifts into place and splits into
// the bytes of each half wave's blocks; the MFMA picks a byte of a word.
template <int MT, int NT>
struct TileShape {
  static constexpr int kWaves = 4, kThreads = kWaves * 64;
  static constexpr int TM = MT * 32, TN = kWaves * NT * 32, kRows = TM + TN;
  static constexpr int kPieces = kRows / 16 / kWaves;  // 1 KB pieces of a stage (16 rows) a wave brings
  static constexpr int kRawPieces = (kRows / 32 + kWaves - 1) / kWaves;  // 1 KB pieces of scales (32 rows)
  static constexpr int kCook = (kRows + kThreads - 1) / kThreads;  // rows whose scales a thread places
  static constexpr int kStage = kRows * 64;
  static constexpr int kRaw = 4 * kStage, kCooked = kRaw + kRawPieces * kWaves * 1024;
  static constexpr int kRowsAt = kCooked + kRows * 16;
  static constexpr int kOutStride = NT * 32 + 4;  // floats
  static constexpr int kBiasAt = kWaves * 32 * kOutStride * 4;
  static constexpr int kLds = kRowsAt + TM * 4;
  static_assert(kRows % (16 * kWaves) == 0 && kBiasAt + TN * 4 <= kRowsAt, "whole pieces; room for the epilogue");
  static_assert(kLds <= 160 * 1024, "LDS of a CU");
};

template <int MT, int NT, int OUT>
__global__ __launch_bounds__(256, 1) void fp4_tile_kernel(Fp4MatmulArgs a, int vec) {
  using S = TileShape<MT, NT>;
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  int* const rows_lds = reinterpret_cast<int*>(lds + S::kRowsAt);
  // the array's offset in the workgroup's LDS
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)lds;
  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l32 = lane & 31, half = lane >> 5;
  Fp4Tile t;
  if (!find_tile<S::TM>(a, (a.N + S::TN - 1) / S::TN, lane, t)) return;
  const int KB = a.K >> 5;
  const int stages = (KB + 3) >> 2;
  const int n0 = t.nt * S::TN;

  for (int i = tid; i < S::TM; i += S::kThreads) rows_lds[i] = routed_row(a, t.p0 + i, t.f);
  __syncthreads();

  // tile row i: X's row of position i (i < TM), then W's row n0 + i - TM; rows
  // past the end read a valid one, whose products are not stored
  auto tile_row = [&](int i) -> size_t {
    if (i < S::TM) {
      const int r = rows_lds[i];
      return r < 0 ? 0 : a.x_div == 1 ? r : r / a.x_div;
    }
    return (size_t)t.e * a.N + min(n0 + i - S::TM, a.N - 1);
  };
  // codes: piece p holds rows 16 p .. + 15; lane l brings row l / 4's LDS slot l % 4
  const int slot = (lane & 3) ^ ((lane >> 3) & 3);
  const uint8_t* src[S::kPieces];
#pragma unroll
  for (int p = 0; p < S::kPieces; p++) {
    const int i = 16 * (wave + S::kWaves * p) + (lane >> 2);
    src[p] = (i < S::TM ? a.x : a.w) + tile_row(i) * KB * 16;
  }
  auto bring = [&](int s, int buf, int p) {
    const int off = min(4 * s + slot, KB - 1) * 16;  // blocks past K: the last one, masked when multiplied
    dma16(src[p] + off, lds0 + buf * S::kStage + (wave + S::kWaves * p) * 1024);
  };
  // scales: piece p holds rows 32 p .. + 31; lane l brings 16-byte piece l % 2 of row l / 2
  const uint8_t* raw_src[S::kRawPieces];  // the group's first, aligned
  int raw_last[S::kRawPieces];            // from it to the piece with the row's last byte
#pragma unroll
  for (int p = 0; p < S::kRawPieces; p++) {
    const int i = min(32 * (wave + S::kWaves * p) + (lane >> 1), S::kRows - 1);
    const uintptr_t row = reinterpret_cast<uintptr_t>(i < S::TM ? a.xs : a.ws) + tile_row(i) * KB;
    raw_src[p] = reinterpret_cast<const uint8_t*>(row & ~(uintptr_t)15);
    raw_last[p] = (int)(((row + KB - 1) & ~(uintptr_t)15) - (row & ~(uintptr_t)15));
  }
  auto bring_scales = [&](int g, int p) {
    dma16(raw_src[p] + min(16 * (g + (lane & 1)), raw_last[p]), lds0 + S::kRaw + (wave + S::kWaves * p) * 1024);
  };
  int shift[S::kCook];
#pragma unroll
  for (int p = 0; p < S::kCook; p++) {
    const int i = min(tid + S::kThreads * p, S::kRows - 1);
    shift[p] = (int)((reinterpret_cast<uintptr_t>(i < S::TM ? a.xs : a.ws) + tile_row(i) * KB) & 15);
  }
  // a group's scale bytes of a row into place: [half wave][8 K steps]
  auto cook = [&]() {
#pragma unroll
    for (int p = 0; p < S::kCook; p++) {
      const int i = tid + S::kThreads * p;
      if (S::kRows % S::kThreads != 0 && i >= S::kRows) break;
      const u32x4_t* q = reinterpret_cast<const u32x4_t*>(lds + S::kRaw + i * 32);
      const u32x4_t lo = q[0], hi = q[1];
      const bool by2 = shift[p] & 8, by1 = shift[p] & 4;
      const uint32_t b[6] = {by2 ? lo.z : lo.x, by2 ? lo.w : lo.y, by2 ? hi.x : lo.z,
                             by2 ? hi.y : lo.w, by2 ? hi.z : hi.x, by2 ? hi.w : hi.y};
      uint32_t d[4];
#pragma unroll
      for (int j = 0; j < 4; j++) {
        const uint32_t d0 = by1 ? b[j + 1] : b[j];
        const uint32_t d1 = by1 ? b[j + 2] : b[j + 1];
        d[j] = __builtin_amdgcn_alignbyte(d1, d0, shift[p] & 3);
      }
      *reinterpret_cast<u32x4_t*>(lds + S::kCooked + i * 16) =
          u32x4_t{__builtin_amdgcn_perm(d[1], d[0], 0x06040200u), __builtin_amdgcn_perm(d[3], d[2], 0x06040200u),
                  __builtin_amdgcn_perm(d[1], d[0], 0x07050301u), __builtin_amdgcn_perm(d[3], d[2], 0x07050301u)};
    }
  };

  const int wr0 = S::TM + wave * NT * 32;
  const int swz = (l32 >> 1) & 3;
  const int off0 = l32 * 64 + ((half ^ swz) << 4), off1 = l32 * 64 + (((2 + half) ^ swz) << 4);

  // The tile with its first MA sub-tiles of routed rows.
  auto run = [&](auto mac) {
    constexpr int MA = decltype(mac)::value;
    v16f acc[NT][MA];
#pragma unroll
    for (int n = 0; n < NT; n++)
#pragma unroll
      for (int m = 0; m < MA; m++)
#pragma unroll
        for (int i = 0; i < 16; i++) acc[n][m][i] = 0.f;
    struct Ops {
      u32x4_t w[NT], x[MA];
    };
    struct Scales {
      uint2 w[NT], x[MA];
    };
    auto read = [&](Ops& o, int buf, int off) {
      const uint8_t* b = lds + buf * S::kStage + off;
#pragma unroll
      for (int n = 0; n < NT; n++) o.w[n] = *reinterpret_cast<const u32x4_t*>(b + (wr0 + 32 * n) * 64);
#pragma unroll
      for (int m = 0; m < MA; m++) o.x[m] = *reinterpret_cast<const u32x4_t*>(b + m * 2048);
    };
    auto read_scales = [&](Scales& c) {
      const uint8_t* b = lds + S::kCooked + l32 * 16 + half * 8;
#pragma unroll
      for (int n = 0; n < NT; n++) c.w[n] = *reinterpret_cast<const uint2*>(b + (wr0 + 32 * n) * 16);
#pragma unroll
      for (int m = 0; m < MA; m++) c.x[m] = *reinterpret_cast<const uint2*>(b + m * 512);
    };
    // K step k (0 .. 7) of the group; `between` follows each MFMA
    auto multiply = [&](const Ops& o, const Scales& c, auto kc, auto between) {
      constexpr int k = decltype(kc)::value;
#pragma unroll
      for (int n = 0; n < NT; n++)
#pragma unroll
        for (int m = 0; m < MA; m++) {
          acc[n][m] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
              fp4_operand(o.w[n]), fp4_operand(o.x[m]), acc[n][m], kFmtFp4, kFmtFp4, k & 3,
              (int)(k < 4 ? c.w[n].x : c.w[n].y), k & 3, (int)(k < 4 ? c.x[m].x : c.x[m].y));
          between(n * MA + m);
        }
    };
    Ops A, Bq;
    Scales sc;

    // Stage s = 4 g + Q, in ring slot Q, with another behind it.  Its first K
    // step is multiplied while the second's operands are read; behind the
    // barrier (every wave has read the slot, and the next stage has arrived)
    // the slot takes stage s + 4 and the next stage's first operands are read
    // while the second step is multiplied.
    auto stage = [&](int g, auto qc) {
      constexpr int Q = decltype(qc)::value;
      constexpr int k = 2 * Q;
      const int s = 4 * g + Q;
      read(Bq, Q, off1);
      pipeline_fence();
      multiply(A, sc, std::integral_constant<int, k>{}, [](int) {});
      if (Q == 3) cook();
      pipeline_fence();
      // under way behind what the next stage needs: two stages, in the second
      // of a group its scales too
      wait_loads<2 * S::kPieces + (Q == 1 ? S::kRawPieces : 0)>();
      asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
      pipeline_fence();
      read(A, (Q + 1) & 3, off0);
      Scales next = sc;
      if (Q == 3) read_scales(next);
      if (Q == 0) {
#pragma unroll
        for (int p = 0; p < S::kRawPieces; p++) bring_scales(g + 1, p);
      }
      pipeline_fence();
      constexpr int kEach = (S::kPieces + NT * MA - 1) / (NT * MA);
      multiply(Bq, sc, std::integral_constant<int, k + 1>{}, [&](int i) {
#pragma unroll
        for (int p = i * kEach; p < (i + 1) * kEach && p < S::kPieces; p++) bring(s + 4, Q, p);
        pipeline_fence();
      });
      sc = next;
    };

#pragma unroll
    for (int p = 0; p < S::kRawPieces; p++) bring_scales(0, p);
#pragma unroll
    for (int s = 0; s < 4; s++)
#pragma unroll
      for (int p = 0; p < S::kPieces; p++) bring(s, s, p);
    wait_loads<4 * S::kPieces < 63 ? 4 * S::kPieces : 63>();
    asm volatile("s_barrier" ::: "memory");
    cook();
    wait_loads<3 * S::kPieces>();
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    read(A, 0, off0);
    read_scales(sc);
    const int last = stages - 1, groups = last >> 2;
    for (int g = 0; g < groups; g++) {
      stage(g, std::integral_constant<int, 0>{});
      stage(g, std::integral_constant<int, 1>{});
      stage(g, std::integral_constant<int, 2>{});
      stage(g, std::integral_constant<int, 3>{});
    }
    if ((last & 3) > 0) stage(groups, std::integral_constant<int, 0>{});
    if ((last & 3) > 1) stage(groups, std::integral_constant<int, 1>{});
    if ((last & 3) > 2) stage(groups, std::integral_constant<int, 2>{});
    // The last stage: blocks past K are taken as zero codes under a finite scale.
    {
      read(Bq, last & 3, off1);
      const int left = KB - 4 * last;
      auto tail = [&](Ops& o, int j) {
        const bool keep = 2 * j + half < left;
        const int k = 2 * (last & 3) + j;
        auto byte = [&](uint2 v) -> uint32_t {
          const uint32_t w = (k < 4 ? v.x : v.y) >> (8 * (k & 3));
          return keep ? w : 0u;
        };
        Scales c;
#pragma unroll
        for (int n = 0; n < NT; n++) c.w[n].x = byte(sc.w[n]);
#pragma unroll
        for (int m = 0; m < MA; m++) {
          c.x[m].x = byte(sc.x[m]);
          o.x[m] = keep ? o.x[m] : u32x4_t{0, 0, 0, 0};
        }
        multiply(o, c, std::integral_constant<int, 0>{}, [](int) {});
      };
      tail(A, 0);
      if (left > 2) tail(Bq, 1);
    }
    wait_loads<0>();  // nothing more comes into LDS
    __syncthreads();

    // Lane (l32, half) holds routed row l32 of each 32 x 32 block and weight rows
    // 8 g + 4 half + i: through LDS, 32 routed rows at a time, so that a store
    // instruction writes whole runs of a row.
    float* const ob = reinterpret_cast<float*>(lds) + wave * 32 * S::kOutStride;
    float* const bias_lds = reinterpret_cast<float*>(lds + S::kBiasAt) + wave * NT * 32;
    const int nw = n0 + wave * NT * 32;
    for (int i = lane; i < NT * 32; i += 64)
      bias_lds[i] = a.bias ? bf16_bits_to_f32(a.bias[(size_t)t.e * a.N + min(nw + i, a.N - 1)]) : 0.f;
#pragma unroll
    for (int m = 0; m < MA; m++) {
#pragma unroll
      for (int n = 0; n < NT; n++)
#pragma unroll
        for (int g = 0; g < 4; g++)
          *reinterpret_cast<f32x4_t*>(ob + l32 * S::kOutStride + 32 * n + 8 * g + 4 * half) =
              f32x4_t{acc[n][m][4 * g], acc[n][m][4 * g + 1], acc[n][m][4 * g + 2], acc[n][m][4 * g + 3]};
      __builtin_amdgcn_wave_barrier();
      constexpr int kChunks = NT * 4;  // 8 columns each
#pragma unroll
      for (int it = 0; it < 32 * kChunks / 64; it++) {
        const int idx = it * 64 + lane;
        const int row = idx / kChunks, cc = idx % kChunks;
        const int r = rows_lds[32 * m + row];
        const int n = nw + 8 * cc;
        float v[8];
        const f32x4_t v0 = *reinterpret_cast<const f32x4_t*>(ob + row * S::kOutStride + 8 * cc);
        const f32x4_t v1 = *reinterpret_cast<const f32x4_t*>(ob + row * S::kOutStride + 8 * cc + 4);
        const f32x4_t b0 = *reinterpret_cast<const f32x4_t*>(bias_lds + 8 * cc);
        const f32x4_t b1 = *reinterpret_cast<const f32x4_t*>(bias_lds + 8 * cc + 4);
#pragma unroll
        for (int i = 0; i < 4; i++) {
          v[i] = v0[i] + b0[i];
          v[4 + i] = v1[i] + b1[i];
        }
        if (r < 0 || n >= a.N) continue;
        if (vec) {
          store8<OUT>(a, r, n, v);
        } else {
#pragma unroll
          for (int i = 0; i < 8; i += 2) store_pair<OUT>(a, r, n + i, v[i], v[i + 1]);
        }
      }
      __builtin_amdgcn_wave_barrier();
    }
  };
  const int subs = (min(t.f - t.p0, S::TM) + 31) >> 5;
  if (MT >= 4 && subs >= 4) run(std::integral_constant<int, MT >= 4 ? 4 : 1>{});
  else if (MT >= 3 && subs == 3) run(std::integral_constant<int, MT >= 3 ? 3 : 1>{});
  else if (MT >= 2 && subs >= 2) run(std::integral_constant<int, MT >= 2 ? 2 : 1>{});
  else run(std::integral_constant<int, 1>{});
}

template <int MT, int NT, int OUT>
hipError_t launch_tiles(const Fp4MatmulArgs& a, hipStream_t stream) {
  using S = TileShape<MT, NT>;
  static DynLdsLimit limit(reinterpret_cast<const void*>(fp4_tile_kernel<MT, NT, OUT>), S::kLds);
  const hipError_t e = limit.ensure();
  if (e != hipSuccess) return e;
  // at most R / TM whole row tiles and one broken one for each expert with rows
  const long long mt = a.offsets ? a.R / S::TM + (long long)min(a.E, a.R) : ((long long)a.R + S::TM - 1) / S::TM;
  const long long tiles = mt * ((a.N + S::TN - 1) / S::TN);
  const long long grid = (tiles + kXcds - 1) / kXcds * kXcds;
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

template <int OUT>
hipError_t launch_out(const Fp4MatmulArgs& a, hipStream_t stream) {
  const long long groups = a.offsets ? min(a.E, a.R) : 1;
  if (a.R <= 16 * groups) return launch_rows<OUT>(a, stream);
  return launch_tiles<4, 3, OUT>(a, stream);
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
