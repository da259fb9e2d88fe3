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
// output written once.  A row belongs to a team of threads, and thread i of it
// holds the chunks i, i + team, ... of eight elements (one or two 16-byte loads
// each): a power of two of lanes up to N = 512, then whole waves, at most eight
// (and two or four chunks a thread beyond N = 4096).  The team follows the row's
// length alone (team_threads), so every kernel here adds a row in the same
// order and the norm of a stored row is the same bits whichever entry point
// takes it.  Sums are fp32: over the thread's elements, the lanes, the waves.
//
// The weights' gradients add over the rows: each workgroup walks the rows
// b, b + grid, ... and keeps its columns' sums in registers, adds its teams' and
// writes them to the workspace once, and a second launch adds the workgroups'
// sums in order (no atomics: the same inputs give the same bits).

#include <type_traits>

#include "kernels.h"
#include "rows.h"

namespace mxfp4 {
namespace {

constexpr int kMaxTeam = 512;
constexpr int kMaxWaves = kMaxTeam / 64;          // of a team
constexpr int kMaxThreads = 1024;                 // of a workgroup, where a thread has one chunk and few registers
constexpr int kMaxWaveTeams = kMaxThreads / 128;  // teams of several waves in a workgroup

// chunks of eight per thread, and the threads of a row's team
int chunks_per_thread(int N) {
  const int chunks = (N + 7) / 8;
  return chunks <= kMaxTeam ? 1 : chunks <= 2 * kMaxTeam ? 2 : 4;
}
int team_threads(int N) {
  const int chunks = (N + 7) / 8, ch = chunks_per_thread(N);
  if (chunks > 64) return ((chunks + ch - 1) / ch + 63) / 64 * 64;
  int t = 1;
  while (t < chunks) t *= 2;
  return t;
}

// f(an element of the row type, the chunks per thread as a constant, whether
// the team is a part of a wave as a constant)
template <typename F>
void with_row_type(bool f32, int N, F f) {
  auto with_chunks = [&](auto elem) {
    if (team_threads(N) < 64) {
      f(elem, std::integral_constant<int, 1>{}, std::true_type{});
      return;
    }
    switch (chunks_per_thread(N)) {
      case 1: f(elem, std::integral_constant<int, 1>{}, std::false_type{}); break;
      case 2: f(elem, std::integral_constant<int, 2>{}, std::false_type{}); break;
      default: f(elem, std::integral_constant<int, 4>{}, std::false_type{}); break;
    }
  };
  if (f32)
    with_chunks(float{});
  else
    with_chunks(uint16_t{});
}

// The teams of a workgroup: blockDim = (threads of a team, teams).  PART: a team
// is a part of a wave (else its number is the same for a whole wave).
template <bool PART>
struct Team {
  int threads, count;  // of a team; teams
  int id, me;          // this thread's team and its place there
  bool tiny;           // rows of fewer than eight elements
  __device__ __forceinline__ explicit Team(int N) : threads(blockDim.x), count(blockDim.y), me(threadIdx.x) {
    id = PART ? (int)threadIdx.y : __builtin_amdgcn_readfirstlane(threadIdx.y);
    tiny = PART && N < 8;
  }
  // the thread's chunk c starts at this element
  __device__ __forceinline__ int at(int c) const { return (me + c * threads) * 8; }
};

template <typename E, bool PART, int CH>
__device__ __forceinline__ void fetch_row(const Team<PART>& team, const E* row, int N, Raw8<E> (&r)[CH]) {
#pragma unroll
  for (int c = 0; c < CH; c++) fetch8(row, team.at(c), N, team.tiny, r[c]);
}
template <typename E, bool PART, int CH>
__device__ __forceinline__ void settle_row(const Team<PART>& team, int N, Raw8<E> (&r)[CH]) {
#pragma unroll
  for (int c = 0; c < CH; c++) settle8(team.at(c), N, r[c]);
}

// the sum over a team's lanes within a wave; every lane receives it
template <bool PART>
__device__ __forceinline__ float lane_sum(const Team<PART>& team, float v) {
  if constexpr (PART) return group_sum_up_to_32(v, team.threads);
  return group_sum<64>(v);
}

// Sums of M values over each team, added lane by lane and then wave by wave;
// every thread receives its team's.  red[.][m] holds value m of each wave, 0
// where the team has fewer waves (its first wave writes those); a buffer is free
// again after the barrier of the next call, so calls take turns between two.
template <bool PART, int M>
__device__ __forceinline__ void row_sum(const Team<PART>& team, float (&v)[M], float (&red)[kMaxWaveTeams][M][kMaxWaves]) {
#pragma unroll
  for (int m = 0; m < M; m++) v[m] = lane_sum(team, v[m]);
  if (PART || team.threads == 64) return;
  const bool spare = team.me < kMaxWaves && team.me >= (team.threads >> 6);
  if ((team.me & 63) == 0 || spare) {
#pragma unroll
    for (int m = 0; m < M; m++) red[team.id][m][spare ? team.me : team.me >> 6] = spare ? 0.f : v[m];
  }
  __syncthreads();
#pragma unroll
  for (int m = 0; m < M; m++) {
    float s = red[team.id][m][0];
#pragma unroll
    for (int w = 1; w < kMaxWaves; w++) s += red[team.id][m][w];
    v[m] = s;
  }
}

__device__ __forceinline__ float rms_scale(float sum, float inv_n, float eps) {
  return rsqrtf(fmaf(sum, inv_n, eps));
}
// sum_n(d w v^) / N from sum_n(d w v).  Where the squares have passed fp32's
// range r is 0 and v^ with it, and the sum of the products, which may have passed
// it as well, is not taken times 0.
__device__ __forceinline__ float unit_mean(float sum, float inv_n, float r) { return r == 0.f ? 0.f : sum * inv_n * r; }

// moe_norm.  Bound by HBM at length: 8192 fp32 rows of 2880 (142 MB) take 26 us,
// 5.4 TB/s, as a copy does; one row takes 2.0 us, the launch and one round trip.
template <typename X, int CH, bool PART>
__global__ __launch_bounds__(kMaxTeam) void norm_kernel(const X* __restrict__ x, const uint16_t* __restrict__ w, int T,
                                                        int N, float inv_n, float eps, uint16_t* __restrict__ xn) {
  __shared__ __align__(16) float red[kMaxWaveTeams][1][kMaxWaves];
  const Team<PART> team(N);
  const int t = blockIdx.x * team.count + team.id;
  const size_t row = (size_t)t * N;
  const int Nt = t < T ? N : 0;
  Raw8<X> xr[CH];
  Raw8<uint16_t> wr[CH];
  fetch_row(team, x + row, Nt, xr);
  fetch_row(team, w, N, wr);
  if (ragged(N)) {
    settle_row(team, Nt, xr);
    settle_row(team, N, wr);
  }
  float s[1] = {0.f};
#pragma unroll
  for (int c = 0; c < CH; c++) {
    float v[8];
    widen8(xr[c], v);
#pragma unroll
    for (int j = 0; j < 8; j++) s[0] = fmaf(v[j], v[j], s[0]);
  }
  row_sum(team, s, red);
  const float r = rms_scale(s[0], inv_n, eps);
#pragma unroll
  for (int c = 0; c < CH; c++) {
    float v[8], wv[8];
    widen8(xr[c], v);
    widen8(wr[c], wv);
#pragma unroll
    for (int j = 0; j < 8; j++) v[j] = v[j] * r * wv[j];
    store8(xn + row, team.at(c), Nt, v);
  }
}

// The block's output.  x_out may be x itself: each element is read and written
// by one thread, in this order (what the row's last chunk reads beside its own
// elements, it drops).  Bound by HBM at length: 8192 x 4 x 2880 (519 MB) take 91
// us, 5.7 TB/s; one token takes 2.9 us.
template <typename X, typename P, int CH, bool PART>
__global__ __launch_bounds__(kMaxTeam) void combine_norm_kernel(const CombineNormArgs a) {
  constexpr int kSlots = CH == 1 ? 4 : CH == 2 ? 2 : 1;  // slots whose rows are under way together
  __shared__ __align__(16) float red[2][kMaxWaveTeams][1][kMaxWaves];
  const int N = a.N, k = a.k;
  const Team<PART> team(N);
  const int t = blockIdx.x * team.count + team.id;
  const int Nt = t < a.T ? N : 0;
  const size_t row = (size_t)t * N;
  const X* x = static_cast<const X*>(a.x) + row;
  X* x_out = static_cast<X*>(a.x_out) + row;
  const P* proj = static_cast<const P*>(a.proj) + row * k;
  Raw8<X> xr[CH];
  Raw8<uint16_t> wp[CH], wn[CH];
  fetch_row(team, x, Nt, xr);
  if (a.w_post) fetch_row(team, a.w_post, N, wp);
  if (a.xn) fetch_row(team, a.w_next, N, wn);
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
      g[u] = 0.f;
      if (q0 + u < k) {
        if (Nt > 0) g[u] = a.gates ? a.gates[(size_t)t * k + q0 + u] : 1.f;
        fetch_row(team, proj + (size_t)(q0 + u) * N, Nt, pr[u]);
      }
    }
    if (ragged(N)) {
#pragma unroll
      for (int u = 0; u < kSlots; u++) settle_row(team, Nt, pr[u]);
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
  if (ragged(N)) {
    settle_row(team, Nt, xr);
    if (a.w_post) settle_row(team, N, wp);
    if (a.xn) settle_row(team, N, wn);
  }
  if (a.w_post) {
#pragma unroll
    for (int c = 0; c < CH; c++)
#pragma unroll
      for (int j = 0; j < 8; j++) s[0] = fmaf(h[c][j], h[c][j], s[0]);
    row_sum(team, s, red[0]);
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
      // rounded to the stream's type before the next norm, which is of the
      // stream as stored: the gradients read it from there, and the separate
      // calls have the same bits
      h[c][j] = rounded(fmaf(a.scale, h[c][j], xv[j]), x);
      s[0] = fmaf(h[c][j], h[c][j], s[0]);
    }
    store8(x_out, team.at(c), Nt, h[c], a.stream);
  }
  if (!a.xn) return;
  row_sum(team, s, red[1]);
  const float r = rms_scale(s[0], a.inv_n, a.eps);
#pragma unroll
  for (int c = 0; c < CH; c++) {
    float wv[8];
    widen8(wn[c], wv);
#pragma unroll
    for (int j = 0; j < 8; j++) h[c][j] = h[c][j] * r * wv[j];
    store8(a.xn + row, team.at(c), Nt, h[c]);
  }
}

// A workgroup's column sums to row blockIdx.x of part: the teams' in order.
template <bool PART, int CH>
__device__ __forceinline__ void store_columns(const Team<PART>& team, float (&dw)[CH][8], float* buf, int N, float* part) {
  if (CH == 1 && team.count > 1) {
    float* mine = buf + (size_t)(team.id * team.threads + team.me) * 8;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 8; j++) mine[j] = dw[0][j];
    __syncthreads();
    if (team.id > 0) return;
    for (int q = 1; q < team.count; q++) {
      mine += team.threads * 8;
#pragma unroll
      for (int j = 0; j < 8; j++) dw[0][j] += mine[j];
    }
  }
#pragma unroll
  for (int c = 0; c < CH; c++) store8(part + (size_t)blockIdx.x * N, team.at(c), N, dw[c]);
}

// Whether a gradient's launch fetches a team's next row ahead: not where a thread
// has four chunks, whose two rows do not fit its registers (norm gradient, 2000
// rows of 16000: 61 us, fetching ahead 181; 4000 of 8000, two chunks: 56 either
// way, and 42 against 46 for the block output's, 1024 x 2 x 8192 bf16).
template <int CH>
constexpr bool kAhead = CH <= 2;

// Gradients of moe_norm.  dx may be dres itself.  8192 rows of 2880 (189 MB): 36
// us, 5.3 TB/s, and 5 us for the column sums' launch; with 1000 rows of fp32 (29
// MB, 10 + 4 us) the round trips of a workgroup's two rows one after the other.
//
// A team's next row is fetched ahead of this row's stores: loads and stores
// complete in the order of their issue, so a load behind the stores would wait
// for them.
template <typename X, int CH, bool PART>
__global__ __launch_bounds__(CH == 1 ? kMaxThreads : kMaxTeam) void norm_backward_kernel(
    const uint16_t* dxn, const X* x, const uint16_t* w, const X* dres, int T, int N, float inv_n, float eps, X* dx,
    float* part) {
  __shared__ __align__(16) float red[2][kMaxWaveTeams][2][kMaxWaves];
  __shared__ __align__(16) float cols[CH == 1 ? kMaxThreads * 8 : 8];
  const Team<PART> team(N);
  const int step = gridDim.x * team.count;
  float dw[CH][8];
  Raw8<uint16_t> wr[CH];
  fetch_row(team, w, N, wr);
#pragma unroll
  for (int c = 0; c < CH; c++)
#pragma unroll
    for (int j = 0; j < 8; j++) dw[c][j] = 0.f;
  Raw8<X> xr[CH], rr[CH];
  Raw8<uint16_t> dr[CH];
  auto fetch = [&](int t) {
    const size_t row = (size_t)t * N;
    const int Nt = t < T ? N : 0;
    fetch_row(team, x + row, Nt, xr);
    fetch_row(team, dxn + row, Nt, dr);
    if (dres) fetch_row(team, dres + row, Nt, rr);
  };
  if constexpr (kAhead<CH>) fetch(blockIdx.x * team.count + team.id);
  if (ragged(N)) settle_row(team, N, wr);
  int parity = 0;
  for (int t0 = blockIdx.x * team.count; t0 < T; t0 += step, parity ^= 1) {
    const int t = t0 + team.id;
    const int Nt = t < T ? N : 0;
    if constexpr (!kAhead<CH>) fetch(t);
    float v[CH][8], d[CH][8], o[CH][8], s[2] = {0.f, 0.f};
    if (ragged(N)) {
      settle_row(team, Nt, xr);
      settle_row(team, Nt, dr);
      if (dres) settle_row(team, Nt, rr);
    }
#pragma unroll
    for (int c = 0; c < CH; c++) {
      float wv[8];
      widen8(xr[c], v[c]);
      widen8(dr[c], d[c]);
      widen8(wr[c], wv);
      if (dres) {
        widen8(rr[c], o[c]);
      } else {
#pragma unroll
        for (int j = 0; j < 8; j++) o[c][j] = 0.f;
      }
#pragma unroll
      for (int j = 0; j < 8; j++) {
        s[0] = fmaf(v[c][j], v[c][j], s[0]);
        s[1] = fmaf(v[c][j], d[c][j] * wv[j], s[1]);
      }
    }
    if constexpr (kAhead<CH>)
      if (t0 + step < T) fetch(t + step);
    row_sum(team, s, red[parity]);
    const float r = rms_scale(s[0], inv_n, eps);
    const float m = unit_mean(s[1], inv_n, r);
#pragma unroll
    for (int c = 0; c < CH; c++) {
      float wv[8];
      widen8(wr[c], wv);
#pragma unroll
      for (int j = 0; j < 8; j++) {
        const float unit = v[c][j] * r;
        dw[c][j] = fmaf(d[c][j], unit, dw[c][j]);
        o[c][j] = fmaf(r, fmaf(-unit, m, d[c][j] * wv[j]), o[c][j]);
      }
      store8(dx + (size_t)t * N, team.at(c), Nt, o[c]);
    }
  }
  if (part) store_columns(team, dw, cols, N, part);
}

// Gradients of moe_combine_norm.  KR > 0: the k <= KR slots' rows stay in
// registers between the combine and the gates' gradients; KR = 0: they are
// read again.  dx may be dx_out itself.  A team's next row is fetched into the
// registers of this row as soon as these have been used, ahead of this row's
// stores (as in norm_backward_kernel); so are its gates.
//
// 8192 x 4 x 2880 (944 MB): 188 us, 5.0 TB/s, and 5 us for the column sums; a
// shorter batch (777 x 3 x 1023, 16 MB, 9.2 + 2.8 us) is bound by one row's chain of
// loads, three sums over the team and stores.  Where the rows are read again they
// come one slot at a time (2048 x 16 x 2880, fp32 proj: 244 us, 3.3 TB/s of what it
// has to move; 2048 x 8 x 2880, held: 102 us, 4.2 TB/s), and four chunks a thread
// spill 233 to 308 registers (500 x 2 x 16000 bf16: 119 us, 1.1 TB/s).
//
// The threads of a workgroup: as many as the registers allow (three waves on a
// SIMD, two with eight slots' rows or more than one chunk a thread).
template <int CH, int KR>
constexpr int kCombineThreads = CH == 1 && KR != 8 ? 768 : kMaxTeam;
template <typename X, typename P, int CH, bool PART, int KR>
__global__ __launch_bounds__((kCombineThreads<CH, KR>)) void combine_norm_backward_kernel(const CombineNormBackwardArgs a) {
  constexpr int KH = KR > 0 ? KR : 1;
  __shared__ __align__(16) float red1[2][kMaxWaveTeams][3][kMaxWaves], red2[2][kMaxWaveTeams][1][kMaxWaves];
  __shared__ __align__(16) float redg[2][kMaxWaveTeams][kMaxTopK][kMaxWaves];
  __shared__ __align__(16) float cols[CH == 1 ? kCombineThreads<CH, KR> * 8 : 8];
  const int N = a.N, k = a.k, T = a.T;
  const Team<PART> team(N);
  const int step = gridDim.x * team.count;
  const bool one_wave = PART || team.threads == 64;
  float dw_post[CH][8], dw_next[CH][8];
  Raw8<uint16_t> wp[CH], wn[CH];
  if (a.w_post) fetch_row(team, a.w_post, N, wp);
  if (a.dxn) fetch_row(team, a.w_next, N, wn);
#pragma unroll
  for (int c = 0; c < CH; c++)
#pragma unroll
    for (int j = 0; j < 8; j++) dw_post[c][j] = dw_next[c][j] = 0.f;
  Raw8<P> pr[KH][CH];
  Raw8<X> gr[CH], xo[CH];
  Raw8<uint16_t> dn[CH];
  float gate_next[KH];
  auto fetch_stream = [&](int t) {
    const size_t row = (size_t)t * N;
    const int Nt = t < T ? N : 0;
    if (a.dx_out) fetch_row(team, static_cast<const X*>(a.dx_out) + row, Nt, gr);
    if (a.dxn) {
      fetch_row(team, static_cast<const X*>(a.x_out) + row, Nt, xo);
      fetch_row(team, a.dxn + row, Nt, dn);
    }
  };
  auto fetch_slot = [&](int t, int q, Raw8<P> (&rows)[CH]) {
    fetch_row(team, static_cast<const P*>(a.proj) + ((size_t)t * k + q) * N, t < T ? N : 0, rows);
  };
  auto gate_of = [&](int t, int q) { return t >= T ? 0.f : a.gates ? a.gates[(size_t)t * k + q] : 1.f; };
  auto fetch_slots = [&](int t) {
    if constexpr (KR > 0) {
#pragma unroll
      for (int q = 0; q < KR; q++) {
        gate_next[q] = q < k ? gate_of(t, q) : 0.f;
        if (q < k) fetch_slot(t, q, pr[q]);
      }
    }
  };
  if constexpr (kAhead<CH>) {
    fetch_slots(blockIdx.x * team.count + team.id);
    fetch_stream(blockIdx.x * team.count + team.id);
  }
  if (ragged(N)) {
    if (a.w_post) settle_row(team, N, wp);
    if (a.dxn) settle_row(team, N, wn);
  }
  // a row's gates' gradients, from its waves' sums behind a barrier
  auto store_dgates = [&](int t, int parity) {
    if (team.me < k && t < T) {
      float d = 0.f;
      for (int w = 0; w < team.threads >> 6; w++) d += redg[parity][team.id][team.me][w];
      a.dgates[(size_t)t * k + team.me] = d;
    }
  };
  const bool sums = a.dxn || a.w_post, shared_dgates = a.dgates && !one_wave;
  int parity = 0, t0 = blockIdx.x * team.count;
  for (; t0 < T; t0 += step, parity ^= 1) {
    const int t = t0 + team.id;
    const int Nt = t < T ? N : 0;
    const size_t row = (size_t)t * N;
    if constexpr (!kAhead<CH>) {
      fetch_slots(t);
      fetch_stream(t);
    }
    float h[CH][8], grad[CH][8], gate[KH], s[3] = {0.f, 0.f, 0.f};
    if (ragged(N)) {
      if constexpr (KR > 0) {
#pragma unroll
        for (int q = 0; q < KR; q++)
          if (q < k) settle_row(team, Nt, pr[q]);
      }
      if (a.dx_out) settle_row(team, Nt, gr);
      if (a.dxn) {
        settle_row(team, Nt, xo);
        settle_row(team, Nt, dn);
      }
    }
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
      for (int q = 0; q < KR; q++) {
        gate[q] = gate_next[q];
        if (q < k) add_slot(gate[q], pr[q]);
      }
    } else {
      for (int q = 0; q < k; q++) {
        fetch_slot(t, q, pr[0]);
        if (ragged(N)) settle_row(team, Nt, pr[0]);
        add_slot(gate_of(t, q), pr[0]);
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
    // the first barrier of this row is also the one behind the last row's
    // dgates
    if (sums)
      row_sum(team, s, red1[parity]);
    else if (shared_dgates)
      __syncthreads();
    if (shared_dgates && t0 >= step) store_dgates(t - step, parity ^ 1);
    if (a.dxn) {
      const float r = rms_scale(s[0], a.inv_n, a.eps);
      const float m = unit_mean(s[1], a.inv_n, r);
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
    if constexpr (kAhead<CH>)
      if (t0 + step < T) fetch_stream(t + step);
    if (a.dx) {
#pragma unroll
      for (int c = 0; c < CH; c++) store8(static_cast<X*>(a.dx) + row, team.at(c), Nt, grad[c]);
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
      row_sum(team, d, red2[parity]);
      const float m = d[0] * a.inv_n;
#pragma unroll
      for (int c = 0; c < CH; c++)
#pragma unroll
        for (int j = 0; j < 8; j++) grad[c][j] = r * fmaf(-(h[c][j] * r), m, grad[c][j]);
    }
    // the slots: dgate = <dh, proj>, dproj = gate * dh
    auto dot_slot = [&](int q, float g, const Raw8<P> (&rows)[CH]) {
      float d = 0.f;
#pragma unroll
      for (int c = 0; c < CH; c++) {
        float p[8];
        widen8(rows[c], p);
#pragma unroll
        for (int j = 0; j < 8; j++) d = fmaf(grad[c][j], p[j], d);
      }
      d = g == 0.f ? 0.f : lane_sum(team, d);
      if (one_wave) {
        if (team.me == 0 && Nt > 0) a.dgates[(size_t)t * k + q] = d;
      } else if ((team.me & 63) == 0) {
        redg[parity][team.id][q][team.me >> 6] = d;
      }
    };
    if (a.dgates) {
      if constexpr (KR > 0) {
#pragma unroll
        for (int q = 0; q < KR; q++)
          if (q < k) dot_slot(q, gate[q], pr[q]);
      } else {
        for (int q = 0; q < k; q++) {
          fetch_slot(t, q, pr[0]);
          if (ragged(N)) settle_row(team, Nt, pr[0]);
          dot_slot(q, gate_of(t, q), pr[0]);
        }
      }
    }
    if constexpr (kAhead<CH>)
      if (t0 + step < T) fetch_slots(t + step);
    if (a.dproj) {
      auto store_slot = [&](int q, float g) {
        P* out = static_cast<P*>(a.dproj) + (row * k + (size_t)q * N);
#pragma unroll
        for (int c = 0; c < CH; c++) {
          float o[8];
#pragma unroll
          for (int j = 0; j < 8; j++) o[j] = g == 0.f ? 0.f : g * grad[c][j];
          store8(out, team.at(c), Nt, o, a.stream);
        }
      };
      if constexpr (KR > 0) {
#pragma unroll
        for (int q = 0; q < KR; q++)
          if (q < k) store_slot(q, gate[q]);
      } else {
        for (int q = 0; q < k; q++) store_slot(q, gate_of(t, q));
      }
    }
  }
  if (shared_dgates) {
    __syncthreads();
    store_dgates(t0 - step + team.id, parity ^ 1);
  }
  if (a.part_post) store_columns(team, dw_post, cols, N, a.part_post);
  if (a.part_next) store_columns(team, dw_next, cols, N, a.part_next);
}

// out[n] = sum_g part[g][n] of at most 256 rows: 16 columns (64 bytes of a row) x
// 64 interleaved groups of rows, a thread's four rows under way together; then
// the four groups of a wave by row swaps, then the waves, all in a fixed order.
constexpr int kSumCols = 16;
constexpr int kSumGroups = 64;
constexpr int kSumDepth = 4;
constexpr int kBackwardGroups = kSumGroups * kSumDepth;  // rows of sums, workgroups of a backward launch
__global__ __launch_bounds__(kSumCols* kSumGroups) void column_sum_kernel(const float* __restrict__ part0, float* out0,
                                                                          const float* __restrict__ part1, float* out1,
                                                                          int G, int N) {
  constexpr int kWaves = kSumCols * kSumGroups / 64;
  __shared__ float red[kWaves][kSumCols];
  const float* part = blockIdx.y ? part1 : part0;
  float* out = blockIdx.y ? out1 : out0;
  const int col = threadIdx.x % kSumCols, grp = threadIdx.x / kSumCols;
  const int n = blockIdx.x * kSumCols + col;
  float s = 0.f;
  if (n < N && G > 0) {
    float v[kSumDepth];
#pragma unroll
    for (int u = 0; u < kSumDepth; u++) v[u] = part[(size_t)min(grp + u * kSumGroups, G - 1) * N + n];
#pragma unroll
    for (int u = 0; u < kSumDepth; u++) s += grp + u * kSumGroups < G ? v[u] : 0.f;
  }
  s = rows_sum(s);
  if ((threadIdx.x & 63) < kSumCols) red[threadIdx.x >> 6][col] = s;
  __syncthreads();
  if (grp == 0 && n < N) {
    s = red[0][col];
#pragma unroll
    for (int w = 1; w < kWaves; w++) s += red[w][col];
    out[n] = s;
  }
}

// Teams and workgroups of a launch, by the rows' number and length alone.
// Forward: workgroups of up to 256 threads.  Backward: up to 256 workgroups, one
// a CU, and then more teams in each, so that the column sums are 256 rows at
// most (two workgroups a CU, block output, 2048 x 4 x 2880 bf16: 48 us; two
// teams in one: 39 us).
constexpr int kForwardThreads = 256;
dim3 forward_block(int N) {
  const int team = team_threads(N);
  return dim3(team, kForwardThreads > team ? kForwardThreads / team : 1);
}
dim3 backward_block(int T, int N, int threads) {
  const int team = team_threads(N);
  const int most = threads > team ? threads / team : 1;
  const int want = (int)(((long long)T + kBackwardGroups - 1) / kBackwardGroups);
  return dim3(team, want < 1 ? 1 : want < most ? want : most);
}
// One chunk a thread and teams of several waves, which wait for each other at
// barriers: 768 or 1024 threads a workgroup (gradients of the block output,
// 8192 x 1 x 2880 bf16: 69 us, with 512 threads 99).  Teams of one wave or less
// do better with 512 (norm gradient, 16384 x 96: 9.1 us, with 1024 threads 10.8;
// block output, 16384 x 4 x 200: 36.5 us, with 768 threads 40.1).
bool many_waves(int N) { return chunks_per_thread(N) == 1 && team_threads(N) > 64; }
int backward_groups(int T, dim3 block) {
  const int groups = (int)(((long long)T + block.y - 1) / block.y);
  return groups < kBackwardGroups ? groups : kBackwardGroups;
}
// rows of one forward launch: a grid holds under 2^32 threads
constexpr int kForwardRows = 1 << 22;
dim3 forward_grid(int T, dim3 block) { return dim3((unsigned)(((long long)T + block.y - 1) / block.y)); }

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
  // a row of column sums for each workgroup, of which there are at most T
  return T > 1 ? (size_t)(T < kBackwardGroups ? T : kBackwardGroups) * N * 4 * weights : 0;
}

hipError_t launch_norm(const void* x, bool x_f32, const uint16_t* w, int T, int N, float eps, uint16_t* xn,
                       hipStream_t stream) {
  const dim3 block = forward_block(N);
  const float inv_n = 1.0f / (float)N;
  hipError_t e = hipSuccess;
  for (int t = 0; t < T && e == hipSuccess; t += kForwardRows) {
    const int rows = T - t < kForwardRows ? T - t : kForwardRows;
    const size_t at = (size_t)t * N;
    with_row_type(x_f32, N, [&](auto elem, auto ch, auto part) {
      using X = decltype(elem);
      hipLaunchKernelGGL((norm_kernel<X, decltype(ch)::value, decltype(part)::value>), forward_grid(rows, block),
                         block, 0, stream, static_cast<const X*>(x) + at, w, rows, N, inv_n, eps, xn + at);
    });
    e = hipGetLastError();
  }
  return e;
}

hipError_t launch_norm_backward(const uint16_t* dxn, const void* x, bool x_f32, const uint16_t* w, const void* dres,
                                int T, int N, float eps, void* dx, float* dw, void* workspace, hipStream_t stream) {
  const dim3 block = backward_block(T, N, many_waves(N) ? kMaxThreads : kMaxTeam);
  const int G = backward_groups(T, block);
  if (G == 0) return launch_column_sums(nullptr, dw, nullptr, nullptr, 0, N, stream);
  float* sums = !dw ? nullptr : G == 1 ? dw : static_cast<float*>(workspace);
  const float inv_n = 1.0f / (float)N;
  with_row_type(x_f32, N, [&](auto elem, auto ch, auto part) {
    using X = decltype(elem);
    hipLaunchKernelGGL((norm_backward_kernel<X, decltype(ch)::value, decltype(part)::value>), dim3(G),
                       block, 0, stream, dxn, static_cast<const X*>(x), w, static_cast<const X*>(dres), T, N, inv_n,
                       eps, static_cast<X*>(dx), sums);
  });
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || G == 1) return e;
  return launch_column_sums(sums, dw, nullptr, nullptr, G, N, stream);
}

// Whether the experts' outputs alone pass the 256 MB cache in front of the HBM:
// then what is not read again at once (x_out, dproj) is stored non-temporally.
// 8192 x 4 x 2880: 95 -> 90 us and 205 -> 200 us; xn and dx are read by the next
// launch and stay ordinary (a router behind a norm of 16384 rows takes 35 us
// after ordinary stores, 41 us after non-temporal ones).
bool streams(int T, int k, int N, bool proj_f32) {
  return (size_t)T * k * N * (proj_f32 ? 4 : 2) > ((size_t)256 << 20);
}

hipError_t launch_combine_norm(CombineNormArgs a, bool x_f32, bool proj_f32, hipStream_t stream) {
  a.stream = streams(a.T, a.k, a.N, proj_f32);
  a.inv_n = 1.0f / (float)a.N;
  const dim3 block = forward_block(a.N);
  const int T = a.T;
  hipError_t e = hipSuccess;
  for (int t = 0; t < T && e == hipSuccess; t += kForwardRows) {
    CombineNormArgs r = a;
    const size_t at = (size_t)t * a.N;
    r.T = T - t < kForwardRows ? T - t : kForwardRows;
    if (r.gates) r.gates += (size_t)t * a.k;
    if (r.xn) r.xn += at;
    const dim3 grid = forward_grid(r.T, block);
    with_row_type(x_f32, a.N, [&](auto elem, auto ch, auto part) {
      using X = decltype(elem);
      constexpr int CH = decltype(ch)::value;
      constexpr bool PART = decltype(part)::value;
      r.x = static_cast<const X*>(a.x) + at;
      r.x_out = static_cast<X*>(a.x_out) + at;
      if (proj_f32) {
        r.proj = static_cast<const float*>(a.proj) + at * a.k;
        hipLaunchKernelGGL((combine_norm_kernel<X, float, CH, PART>), grid, block, 0, stream, r);
      } else {
        r.proj = static_cast<const uint16_t*>(a.proj) + at * a.k;
        hipLaunchKernelGGL((combine_norm_kernel<X, uint16_t, CH, PART>), grid, block, 0, stream, r);
      }
    });
    e = hipGetLastError();
  }
  return e;
}

hipError_t launch_combine_norm_backward(CombineNormBackwardArgs a, bool x_f32, bool proj_f32, float* dw_post,
                                        float* dw_next, void* workspace, hipStream_t stream) {
  // the slots' rows held in registers: at most 64 values a thread
  const int ch = chunks_per_thread(a.N);
  const int most = ch == 1 ? 8 : ch == 2 ? 4 : 0, few = most / 2;
  const int held = a.k <= few ? few : a.k <= most ? most : 0;
  const dim3 block = backward_block(a.T, a.N, many_waves(a.N) && held != 8 ? kCombineThreads<1, 0> : kMaxTeam);
  const int G = backward_groups(a.T, block);
  if (G == 0) return launch_column_sums(nullptr, dw_post, nullptr, dw_next, 0, a.N, stream);
  a.stream = streams(a.T, a.k, a.N, proj_f32);
  float* ws = static_cast<float*>(workspace);
  a.part_post = !dw_post ? nullptr : G == 1 ? dw_post : ws;
  a.part_next = !dw_next ? nullptr : G == 1 ? dw_next : ws + (size_t)G * a.N;
  a.inv_n = 1.0f / (float)a.N;
  const dim3 grid(G);
  with_row_type(x_f32, a.N, [&](auto elem, auto ch, auto part) {
    using X = decltype(elem);
    constexpr int CH = decltype(ch)::value;
    constexpr bool PART = decltype(part)::value;
    constexpr int most = CH == 1 ? 8 : CH == 2 ? 4 : 0, few = most / 2;
    auto with_proj = [&](auto pelem) {
      using P = decltype(pelem);
      auto launch = [&](auto rows) {
        hipLaunchKernelGGL((combine_norm_backward_kernel<X, P, CH, PART, decltype(rows)::value>), grid, block, 0,
                           stream, a);
      };
      if (a.k <= few)
        launch(std::integral_constant<int, few>{});
      else if (a.k <= most)
        launch(std::integral_constant<int, most>{});
      else
        launch(std::integral_constant<int, 0>{});
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
