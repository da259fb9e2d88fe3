// The root-mean-square norms before and after the expert block, for gfx950:
// the input norm of the router and the experts, and the block's output --
// combine, output norm, residual scale, residual sum and the next block's
// input norm in one pass -- with their gradients.
//
//   norm(v, w)[n] = v[n] * r * w[n],   r = (sum_n v[n]^2 / N + eps)^(-1/2)
//   moe_norm          xn = norm(x, w)
//   moe_combine_norm  h = sum_s gates[s] * proj[s];  u = norm(h, w_post) or h
//                     x_out = x + scale * u;         xn = norm(x_out, w_next)
//
// The gradient of norm at v, for the gradient d of its result, with
// v^ = v * r:  dv = r * (d w - v^ * sum_n(d w v^) / N),  dw = sum_t d v^.
//
// All of it is a stream through HBM with one to three row sums in the middle.
// A row stays in registers between them, so each input is read once and each
// output written once: a row belongs to a workgroup of NT threads (a multiple
// of 64, at most 512), and thread i holds the chunks i, i + NT, ... of eight
// elements (one or two 16-byte loads each).  NT follows the row's length alone
// (row_threads), so every kernel here adds a row in the same order and the
// norm of a stored row is the same bits whichever entry point takes it.
// Sums are fp32: over the thread's elements, the wave's lanes, the waves.
//
// The weights' gradients add over the rows: each workgroup walks the rows
// b, b + grid, ... and keeps its columns' sums in registers, writes them to
// the workspace once, and a second launch adds the workgroups' sums in order
// (no atomics: the same inputs give the same bits).

#include <type_traits>

#include "kernels.h"
#include "rows.h"

namespace mxfp4 {
namespace {

constexpr int kMaxRowThreads = 512;
constexpr int kMaxWaves = kMaxRowThreads / 64;

// chunks of eight per thread, and the threads of a row
int row_chunks_per_thread(int N) {
  const int chunks = (N + 7) / 8;
  return chunks <= kMaxRowThreads ? 1 : chunks <= 2 * kMaxRowThreads ? 2 : 4;
}
int row_threads(int N) {
  const int chunks = (N + 7) / 8, ch = row_chunks_per_thread(N);
  return ((chunks + ch - 1) / ch + 63) / 64 * 64;
}

// f(an element of the row type, the chunks per thread as a constant)
template <typename F>
void with_row_type(bool f32, int N, F f) {
  auto with_chunks = [&](auto elem) {
    switch (row_chunks_per_thread(N)) {
      case 1: f(elem, std::integral_constant<int, 1>{}); break;
      case 2: f(elem, std::integral_constant<int, 2>{}); break;
      default: f(elem, std::integral_constant<int, 4>{}); break;
    }
  };
  if (f32)
    with_chunks(float{});
  else
    with_chunks(uint16_t{});
}

// Sums of M values over the workgroup, added lane by lane and then wave by
// wave; every thread receives them.  red[m] holds value m of each wave, 0
// where the row has fewer waves (wave 0 writes those); a buffer is free again after the
// barrier of the next call, so calls take turns between two.
template <int M>
__device__ __forceinline__ void row_sum(float (&v)[M], float (&red)[M][kMaxWaves]) {
#pragma unroll
  for (int m = 0; m < M; m++) v[m] = group_sum<64>(v[m]);
  if (blockDim.x == 64) return;
  const int lane = threadIdx.x & 63;
  const bool spare = threadIdx.x < kMaxWaves && threadIdx.x >= (blockDim.x >> 6);
  if (lane == 0 || spare) {
#pragma unroll
    for (int m = 0; m < M; m++) red[m][spare ? lane : threadIdx.x >> 6] = spare ? 0.f : v[m];
  }
  __syncthreads();
#pragma unroll
  for (int m = 0; m < M; m++) {
    float s = red[m][0];
#pragma unroll
    for (int w = 1; w < kMaxWaves; w++) s += red[m][w];
    v[m] = s;
  }
}

__device__ __forceinline__ float rms_scale(float sum, float inv_n, float eps) {
  return rsqrtf(fmaf(sum, inv_n, eps));
}

// a thread's chunks of a row: c = 0 .. CH - 1 at element (thread + c * threads) * 8
__device__ __forceinline__ int chunk_at(int c) { return (threadIdx.x + c * blockDim.x) * 8; }

template <typename E, int CH>
__device__ __forceinline__ void fetch_row(const E* row, int N, Raw8<E> (&r)[CH]) {
#pragma unroll
  for (int c = 0; c < CH; c++) fetch8(row + chunk_at(c), N - chunk_at(c), r[c]);
}

template <typename X, int CH>
__global__ __launch_bounds__(kMaxRowThreads) void norm_kernel(const X* __restrict__ x, const uint16_t* __restrict__ w,
                                                              int N, float inv_n, float eps,
                                                              uint16_t* __restrict__ xn) {
  __shared__ __align__(16) float red[1][kMaxWaves];
  const size_t row = (size_t)blockIdx.x * N;
  Raw8<X> xr[CH];
  Raw8<uint16_t> wr[CH];
  fetch_row(x + row, N, xr);
  fetch_row(w, N, wr);
  float s[1] = {0.f};
#pragma unroll
  for (int c = 0; c < CH; c++) {
    float v[8];
    widen8(xr[c], v);
#pragma unroll
    for (int j = 0; j < 8; j++) s[0] = fmaf(v[j], v[j], s[0]);
  }
  row_sum(s, red);
  const float r = rms_scale(s[0], inv_n, eps);
#pragma unroll
  for (int c = 0; c < CH; c++) {
    float v[8], wv[8];
    widen8(xr[c], v);
    widen8(wr[c], wv);
#pragma unroll
    for (int j = 0; j < 8; j++) v[j] = v[j] * r * wv[j];
    store8(xn + row + chunk_at(c), N - chunk_at(c), v);
  }
}

// The block's output.  x_out may be x itself: each element is read and written
// by one thread, in this order.
template <typename X, typename P, int CH>
__global__ __launch_bounds__(kMaxRowThreads) void combine_norm_kernel(const CombineNormArgs a) {
  constexpr int kSlots = CH == 1 ? 4 : CH == 2 ? 2 : 1;  // slots whose rows are under way together
  __shared__ __align__(16) float red[2][1][kMaxWaves];
  const int N = a.N, k = a.k;
  const size_t t = blockIdx.x, row = t * N;
  const X* x = static_cast<const X*>(a.x) + row;
  X* x_out = static_cast<X*>(a.x_out) + row;
  const P* proj = static_cast<const P*>(a.proj) + row * k;
  Raw8<X> xr[CH];
  Raw8<uint16_t> wp[CH], wn[CH];
  fetch_row(x, N, xr);
  if (a.w_post) fetch_row(a.w_post, N, wp);
  if (a.xn) fetch_row(a.w_next, N, wn);
  float h[CH][8], s[1] = {0.f};
#pragma unroll
  for (int c = 0; c < CH; c++)
#pragma unroll
    for (int j = 0; j < 8; j++) h[c][j] = 0.f;
  for (int q0 = 0; q0 < k; q0 += kSlots) {
    Raw8<P> pr[kSlots][CH];
    float g[kSlots];
#pragma unroll
    for (int u = 0; u < kSlots; u++) {
      const int q = min(q0 + u, k - 1);
      g[u] = q0 + u >= k ? 0.f : a.gates ? a.gates[t * k + q] : 1.f;
      fetch_row(proj + (size_t)q * N, N, pr[u]);
    }
#pragma unroll
    for (int u = 0; u < kSlots; u++) {
      if (g[u] == 0.f) continue;
#pragma unroll
      for (int c = 0; c < CH; c++) {
        float p[8];
        widen8(pr[u][c], p);
#pragma unroll
        for (int j = 0; j < 8; j++) h[c][j] = fmaf(g[u], p[j], h[c][j]);
      }
    }
  }
  if (a.w_post) {
#pragma unroll
    for (int c = 0; c < CH; c++)
#pragma unroll
      for (int j = 0; j < 8; j++) s[0] = fmaf(h[c][j], h[c][j], s[0]);
    row_sum(s, red[0]);
    const float r = rms_scale(s[0], a.inv_n, a.eps);
#pragma unroll
    for (int c = 0; c < CH; c++) {
      float wv[8];
      widen8(wp[c], wv);
#pragma unroll
      for (int j = 0; j < 8; j++) h[c][j] = h[c][j] * r * wv[j];
    }
  }
  s[0] = 0.f;
#pragma unroll
  for (int c = 0; c < CH; c++) {
    float xv[8];
    widen8(xr[c], xv);
#pragma unroll
    for (int j = 0; j < 8; j++) {
      h[c][j] = rounded(fmaf(a.scale, h[c][j], xv[j]), x);
      s[0] = fmaf(h[c][j], h[c][j], s[0]);
    }
    store8(x_out + chunk_at(c), N - chunk_at(c), h[c]);
  }
  if (!a.xn) return;
  row_sum(s, red[1]);
  const float r = rms_scale(s[0], a.inv_n, a.eps);
#pragma unroll
  for (int c = 0; c < CH; c++) {
    float wv[8];
    widen8(wn[c], wv);
#pragma unroll
    for (int j = 0; j < 8; j++) h[c][j] = h[c][j] * r * wv[j];
    store8(a.xn + row + chunk_at(c), N - chunk_at(c), h[c]);
  }
}

// Gradients of moe_norm.  dx may be dres itself.  The loads of a workgroup's
// next row are issued before the sums of this one.
template <typename X, int CH>
__global__ __launch_bounds__(kMaxRowThreads) void norm_backward_kernel(const uint16_t* dxn, const X* x,
                                                                       const uint16_t* w, const X* dres, int T, int N,
                                                                       float inv_n, float eps, X* dx, float* part) {
  __shared__ __align__(16) float red[2][2][kMaxWaves];
  float dw[CH][8];
  Raw8<uint16_t> wr[CH];
  fetch_row(w, N, wr);
#pragma unroll
  for (int c = 0; c < CH; c++)
#pragma unroll
    for (int j = 0; j < 8; j++) dw[c][j] = 0.f;
  Raw8<X> x_next[CH], r_next[CH];
  Raw8<uint16_t> d_next[CH];
  auto fetch = [&](int t) {
    const size_t row = (size_t)t * N;
    fetch_row(x + row, N, x_next);
    fetch_row(dxn + row, N, d_next);
    if (dres) fetch_row(dres + row, N, r_next);
  };
  fetch(blockIdx.x);
  int parity = 0;
  for (int t = blockIdx.x; t < T; t += gridDim.x, parity ^= 1) {
    Raw8<X> rr[CH];
    float v[CH][8], d[CH][8], s[2] = {0.f, 0.f};
#pragma unroll
    for (int c = 0; c < CH; c++) {
      float wv[8];
      widen8(x_next[c], v[c]);
      widen8(d_next[c], d[c]);
      widen8(wr[c], wv);
      rr[c] = r_next[c];
#pragma unroll
      for (int j = 0; j < 8; j++) {
        s[0] = fmaf(v[c][j], v[c][j], s[0]);
        s[1] = fmaf(v[c][j], d[c][j] * wv[j], s[1]);
      }
    }
    if (t + (int)gridDim.x < T) fetch(t + gridDim.x);
    row_sum(s, red[parity]);
    const float r = rms_scale(s[0], inv_n, eps);
    const float m = s[1] * inv_n * r;
#pragma unroll
    for (int c = 0; c < CH; c++) {
      float o[8], wv[8];
      widen8(wr[c], wv);
      if (dres) {
        widen8(rr[c], o);
      } else {
#pragma unroll
        for (int j = 0; j < 8; j++) o[j] = 0.f;
      }
#pragma unroll
      for (int j = 0; j < 8; j++) {
        const float unit = v[c][j] * r;
        dw[c][j] = fmaf(d[c][j], unit, dw[c][j]);
        o[j] = fmaf(r, fmaf(-unit, m, d[c][j] * wv[j]), o[j]);
      }
      store8(dx + (size_t)t * N + chunk_at(c), N - chunk_at(c), o);
    }
  }
  if (part) {
#pragma unroll
    for (int c = 0; c < CH; c++) store8(part + (size_t)blockIdx.x * N + chunk_at(c), N - chunk_at(c), dw[c]);
  }
}

// Gradients of moe_combine_norm.  KR > 0: the k <= KR slots' rows stay in
// registers between the combine and the gates' gradients; KR = 0: they are
// read again.  dx may be dx_out itself.
//
// A workgroup's next row is fetched into the registers of this row as soon as
// these have been used, ahead of this row's stores: loads and stores complete
// in the order of their issue, so a load behind the stores would wait for them.
template <typename X, typename P, int CH, int KR>
__global__ __launch_bounds__(kMaxRowThreads) void combine_norm_backward_kernel(const CombineNormBackwardArgs a) {
  constexpr int KH = KR > 0 ? KR : 1;
  __shared__ __align__(16) float red1[2][3][kMaxWaves], red2[2][1][kMaxWaves], redg[2][kMaxTopK][kMaxWaves];
  const int N = a.N, k = a.k;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
  float dw_post[CH][8], dw_next[CH][8];
  Raw8<uint16_t> wp[CH], wn[CH];
  if (a.w_post) fetch_row(a.w_post, N, wp);
  if (a.dxn) fetch_row(a.w_next, N, wn);
#pragma unroll
  for (int c = 0; c < CH; c++)
#pragma unroll
    for (int j = 0; j < 8; j++) dw_post[c][j] = dw_next[c][j] = 0.f;
  Raw8<P> pr[KH][CH];
  Raw8<X> gr[CH], xo[CH];
  Raw8<uint16_t> dn[CH];
  auto fetch_stream = [&](int t) {
    const size_t row = (size_t)t * N;
    if (a.dx_out) fetch_row(static_cast<const X*>(a.dx_out) + row, N, gr);
    if (a.dxn) {
      fetch_row(static_cast<const X*>(a.x_out) + row, N, xo);
      fetch_row(a.dxn + row, N, dn);
    }
  };
  auto fetch_slot = [&](int t, int q, Raw8<P> (&rows)[CH]) {
    fetch_row(static_cast<const P*>(a.proj) + ((size_t)t * k + q) * N, N, rows);
  };
  auto fetch_slots = [&](int t) {
    if constexpr (KR > 0) {
#pragma unroll
      for (int q = 0; q < KR; q++)
        if (q < k) fetch_slot(t, q, pr[q]);
    }
  };
  fetch_slots(blockIdx.x);
  fetch_stream(blockIdx.x);
  int parity = 0;
  for (int t = blockIdx.x; t < a.T; t += gridDim.x, parity ^= 1) {
    const bool more = t + (int)gridDim.x < a.T;
    const size_t row = (size_t)t * N;
    const float* gates = a.gates ? a.gates + (size_t)t * k : nullptr;
    float h[CH][8], grad[CH][8], s[3] = {0.f, 0.f, 0.f};
#pragma unroll
    for (int c = 0; c < CH; c++)
#pragma unroll
      for (int j = 0; j < 8; j++) h[c][j] = 0.f;
    auto add_slot = [&](float g, const Raw8<P> (&rows)[CH]) {
      if (g == 0.f) return;
#pragma unroll
      for (int c = 0; c < CH; c++) {
        float p[8];
        widen8(rows[c], p);
#pragma unroll
        for (int j = 0; j < 8; j++) h[c][j] = fmaf(g, p[j], h[c][j]);
      }
    };
    if constexpr (KR > 0) {
#pragma unroll
      for (int q = 0; q < KR; q++)
        if (q < k) add_slot(gates ? gates[q] : 1.f, pr[q]);
    } else {
      for (int q = 0; q < k; q++) {
        fetch_slot(t, q, pr[0]);
        add_slot(gates ? gates[q] : 1.f, pr[0]);
      }
    }
    // the gradient at x_out: the stream's own and the next norm's
#pragma unroll
    for (int c = 0; c < CH; c++) {
      if (a.dx_out) {
        widen8(gr[c], grad[c]);
      } else {
#pragma unroll
        for (int j = 0; j < 8; j++) grad[c][j] = 0.f;
      }
      if (a.dxn) {
        float wv[8], xv[8], dv[8];
        widen8(xo[c], xv);
        widen8(dn[c], dv);
        widen8(wn[c], wv);
#pragma unroll
        for (int j = 0; j < 8; j++) {
          s[0] = fmaf(xv[j], xv[j], s[0]);
          s[1] = fmaf(xv[j], dv[j] * wv[j], s[1]);
        }
      }
#pragma unroll
      for (int j = 0; j < 8; j++) s[2] = fmaf(h[c][j], h[c][j], s[2]);
    }
    if (a.dxn || a.w_post) row_sum(s, red1[parity]);
    if (a.dxn) {
      const float r = rms_scale(s[0], a.inv_n, a.eps);
      const float m = s[1] * a.inv_n * r;
#pragma unroll
      for (int c = 0; c < CH; c++) {
        float wv[8], xv[8], dv[8];
        widen8(xo[c], xv);
        widen8(dn[c], dv);
        widen8(wn[c], wv);
#pragma unroll
        for (int j = 0; j < 8; j++) {
          const float unit = xv[j] * r;
          dw_next[c][j] = fmaf(dv[j], unit, dw_next[c][j]);
          grad[c][j] = fmaf(r, fmaf(-unit, m, dv[j] * wv[j]), grad[c][j]);
        }
      }
    }
    if (more) fetch_stream(t + gridDim.x);
    if (a.dx) {
#pragma unroll
      for (int c = 0; c < CH; c++)
        store8(static_cast<X*>(a.dx) + row + chunk_at(c), N - chunk_at(c), grad[c]);
    }
    // through the residual scale and the output norm: grad becomes dh
#pragma unroll
    for (int c = 0; c < CH; c++)
#pragma unroll
      for (int j = 0; j < 8; j++) grad[c][j] *= a.scale;
    if (a.w_post) {
      const float r = rms_scale(s[2], a.inv_n, a.eps);
      float d[1] = {0.f};
#pragma unroll
      for (int c = 0; c < CH; c++) {
        float wv[8];
        widen8(wp[c], wv);
#pragma unroll
        for (int j = 0; j < 8; j++) {
          const float unit = h[c][j] * r;
          dw_post[c][j] = fmaf(grad[c][j], unit, dw_post[c][j]);
          grad[c][j] *= wv[j];
          d[0] = fmaf(grad[c][j], unit, d[0]);
        }
      }
      row_sum(d, red2[parity]);
      const float m = d[0] * a.inv_n;
#pragma unroll
      for (int c = 0; c < CH; c++)
#pragma unroll
        for (int j = 0; j < 8; j++) grad[c][j] = r * fmaf(-(h[c][j] * r), m, grad[c][j]);
    }
    // the slots: dgate = <dh, proj>, dproj = gate * dh
    auto dot_slot = [&](int q, const Raw8<P> (&rows)[CH]) {
      float d = 0.f;
#pragma unroll
      for (int c = 0; c < CH; c++) {
        float p[8];
        widen8(rows[c], p);
#pragma unroll
        for (int j = 0; j < 8; j++) d = fmaf(grad[c][j], p[j], d);
      }
      d = group_sum<64>(d);
      if (lane == 0) redg[parity][q][wave] = d;
    };
    if (a.dgates) {
      if constexpr (KR > 0) {
#pragma unroll
        for (int q = 0; q < KR; q++)
          if (q < k) dot_slot(q, pr[q]);
      } else {
        for (int q = 0; q < k; q++) {
          fetch_slot(t, q, pr[0]);
          dot_slot(q, pr[0]);
        }
      }
    }
    if (more) fetch_slots(t + gridDim.x);
    if (a.dproj) {
      for (int q = 0; q < k; q++) {
        const float g = gates ? gates[q] : 1.f;
        P* out = static_cast<P*>(a.dproj) + (row * k + (size_t)q * N);
#pragma unroll
        for (int c = 0; c < CH; c++) {
          float o[8];
#pragma unroll
          for (int j = 0; j < 8; j++) o[j] = g * grad[c][j];
          store8(out + chunk_at(c), N - chunk_at(c), o);
        }
      }
    }
    if (a.dgates) {
      __syncthreads();
      if ((int)threadIdx.x < k) {
        float d = 0.f;
        for (int w = 0; w < waves; w++) d += redg[parity][threadIdx.x][w];
        a.dgates[(size_t)t * k + threadIdx.x] = gates[threadIdx.x] == 0.f ? 0.f : d;
      }
    }
  }
#pragma unroll
  for (int c = 0; c < CH; c++) {
    const size_t at = (size_t)blockIdx.x * N + chunk_at(c);
    if (a.part_post) store8(a.part_post + at, N - chunk_at(c), dw_post[c]);
    if (a.part_next) store8(a.part_next + at, N - chunk_at(c), dw_next[c]);
  }
}

// out[n] = sum_g part[g][n]: 16 columns (64 bytes of a row) x 64 interleaved
// groups of rows, each added in order (eight loads under way), then the groups
// in order.
constexpr int kSumCols = 16;
constexpr int kSumGroups = 64;
constexpr int kSumDepth = 8;
__global__ __launch_bounds__(kSumCols* kSumGroups) void column_sum_kernel(const float* __restrict__ part0, float* out0,
                                                                          const float* __restrict__ part1, float* out1,
                                                                          int G, int N) {
  __shared__ float red[kSumGroups][kSumCols + 1];
  const float* part = blockIdx.y ? part1 : part0;
  float* out = blockIdx.y ? out1 : out0;
  const int col = threadIdx.x % kSumCols, grp = threadIdx.x / kSumCols;
  const int n = blockIdx.x * kSumCols + col;
  float s = 0.f;
  if (n < N) {
    for (int g = grp; g < G; g += kSumGroups * kSumDepth) {
      float v[kSumDepth];
#pragma unroll
      for (int u = 0; u < kSumDepth; u++) {
        const int gu = g + u * kSumGroups;
        v[u] = part[(size_t)min(gu, G - 1) * N + n];
      }
#pragma unroll
      for (int u = 0; u < kSumDepth; u++) s += g + u * kSumGroups < G ? v[u] : 0.f;
    }
  }
  red[grp][col] = s;
  __syncthreads();
  if (grp == 0 && n < N) {
    float v = red[0][col];
#pragma unroll
    for (int g = 1; g < kSumGroups; g++) v += red[g][col];
    out[n] = v;
  }
}

// The workgroups of a backward launch, by the rows alone: enough to fill the
// 256 CUs twice, few enough that their column sums stay small beside the rows.
constexpr int kBackwardGroups = 512;
int backward_groups(int T) { return T < kBackwardGroups ? T : kBackwardGroups; }

// the outputs that are wanted (not NULL); G = 0 rows of sums: zeros
hipError_t launch_column_sums(const float* part0, float* out0, const float* part1, float* out1, int G, int N,
                              hipStream_t stream) {
  if (!out0) {
    part0 = part1, out0 = out1;
    out1 = nullptr;
  }
  if (!out0) return hipSuccess;
  hipLaunchKernelGGL(column_sum_kernel, dim3((unsigned)((N + kSumCols - 1) / kSumCols), out1 ? 2 : 1),
                     dim3(kSumCols * kSumGroups), 0, stream, part0, out0, part1, out1, G, N);
  return hipGetLastError();
}

}  // namespace

size_t norm_backward_workspace_bytes(int T, int N, int weights) {
  return T > 1 ? (size_t)backward_groups(T) * N * 4 * weights : 0;
}

hipError_t launch_norm(const void* x, bool x_f32, const uint16_t* w, int T, int N, float eps, uint16_t* xn,
                       hipStream_t stream) {
  const dim3 grid(T), block(row_threads(N));
  const float inv_n = 1.0f / (float)N;
  with_row_type(x_f32, N, [&](auto elem, auto ch) {
    using X = decltype(elem);
    hipLaunchKernelGGL((norm_kernel<X, decltype(ch)::value>), grid, block, 0, stream, static_cast<const X*>(x), w, N,
                       inv_n, eps, xn);
  });
  return hipGetLastError();
}

hipError_t launch_norm_backward(const uint16_t* dxn, const void* x, bool x_f32, const uint16_t* w, const void* dres,
                                int T, int N, float eps, void* dx, float* dw, void* workspace, hipStream_t stream) {
  const int G = backward_groups(T);
  if (G == 0) return launch_column_sums(nullptr, dw, nullptr, nullptr, 0, N, stream);
  float* part = !dw ? nullptr : G == 1 ? dw : static_cast<float*>(workspace);
  const dim3 grid(G), block(row_threads(N));
  const float inv_n = 1.0f / (float)N;
  with_row_type(x_f32, N, [&](auto elem, auto ch) {
    using X = decltype(elem);
    hipLaunchKernelGGL((norm_backward_kernel<X, decltype(ch)::value>), grid, block, 0, stream, dxn,
                       static_cast<const X*>(x), w, static_cast<const X*>(dres), T, N, inv_n, eps,
                       static_cast<X*>(dx), part);
  });
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || G == 1 || !dw) return e;
  return launch_column_sums(part, dw, nullptr, nullptr, G, N, stream);
}

hipError_t launch_combine_norm(CombineNormArgs a, bool x_f32, bool proj_f32, int T, hipStream_t stream) {
  const dim3 grid(T), block(row_threads(a.N));
  a.inv_n = 1.0f / (float)a.N;
  with_row_type(x_f32, a.N, [&](auto elem, auto ch) {
    using X = decltype(elem);
    if (proj_f32)
      hipLaunchKernelGGL((combine_norm_kernel<X, float, decltype(ch)::value>), grid, block, 0, stream, a);
    else
      hipLaunchKernelGGL((combine_norm_kernel<X, uint16_t, decltype(ch)::value>), grid, block, 0, stream, a);
  });
  return hipGetLastError();
}

hipError_t launch_combine_norm_backward(CombineNormBackwardArgs a, bool x_f32, bool proj_f32, float* dw_post,
                                        float* dw_next, void* workspace, hipStream_t stream) {
  const int G = backward_groups(a.T);
  if (G == 0) return launch_column_sums(nullptr, dw_post, nullptr, dw_next, 0, a.N, stream);
  const size_t part = (size_t)G * a.N;
  float* ws = static_cast<float*>(workspace);
  a.part_post = !dw_post ? nullptr : G == 1 ? dw_post : ws;
  a.part_next = !dw_next ? nullptr : G == 1 ? dw_next : ws + part;
  a.inv_n = 1.0f / (float)a.N;
  const dim3 grid(G), block(row_threads(a.N));
  with_row_type(x_f32, a.N, [&](auto elem, auto ch) {
    using X = decltype(elem);
    constexpr int CH = decltype(ch)::value;
    // the slots' rows held in registers: at most 64 values a thread
    constexpr int KR = CH == 1 ? 8 : CH == 2 ? 4 : 0;
    constexpr int KS = CH == 1 ? 4 : CH == 2 ? 2 : 0;
    auto with_proj = [&](auto pelem) {
      using P = decltype(pelem);
      if (a.k <= KS)
        hipLaunchKernelGGL((combine_norm_backward_kernel<X, P, CH, KS>), grid, block, 0, stream, a);
      else if (a.k <= KR)
        hipLaunchKernelGGL((combine_norm_backward_kernel<X, P, CH, KR>), grid, block, 0, stream, a);
      else
        hipLaunchKernelGGL((combine_norm_backward_kernel<X, P, CH, 0>), grid, block, 0, stream, a);
    };
    if (proj_f32)
      with_proj(float{});
    else
      with_proj(uint16_t{});
  });
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || G == 1) return e;
  return launch_column_sums(a.part_post, dw_post, a.part_next, dw_next, G, a.N, stream);
}

}  // namespace mxfp4
