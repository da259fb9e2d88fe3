// The routing's balance loss and per-expert counts, and the gradient of the
// router's logits, for gfx950.
//
// With p[t] the softmax of token t's E logits and z[t] their log-sum-exp, for
// a sequence s of n_s counted tokens whose slots chose expert e c[s, e] times:
//
//   balance = mean over the non-empty sequences of
//             E * sum_e (c[s, e] / (k n_s)) * (sum_{t in s} p[t, e] / n_s)
//   z loss  = mean over the counted tokens of z[t]^2
//
// c does not depend on the logits by any derivative, so with a = E dbalance /
// (S' k n_s^2) (S' sequences, n tokens in all) and b = 2 dz / n
//
//   dlogits[t, e] = p[t, e] (a (c[s, e] - sum_j p[t, j] c[s, j]) + b z[t])
//                   + sum over the slots q of t that chose e of
//                     g[q] (dg[q] - sum_r g[r] dg[r])
//
// (the last sum: the gates are a softmax over the chosen logits).  The mean of
// c over the experts is taken off first, which leaves the value as it is and
// keeps the difference exact where the load is even.
//
// A token is counted when it lies in a sequence, has a slot with a valid
// expert and a logit above -inf; any other token's logits reach no sum.
//
// Layout: a token belongs to a group of L lanes (a power of two), each holding
// eight neighbouring experts (one 16-byte load), so 64 / L tokens run in a wave
// and a token's maximum and sum take log2(L) lane exchanges.

#include <type_traits>

#include "kernels.h"
#include "rows.h"

namespace mxfp4 {
namespace {

constexpr int kThreads = 256;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

template <int L>
__device__ __forceinline__ bool group_any(bool p) {
  const uint64_t m = __ballot(p);
  if constexpr (L == 64) return m != 0;
  const int base = (threadIdx.x & 63) & ~(L - 1);
  return ((m >> base) & ((1ull << (L & 63)) - 1)) != 0;
}

// a lane's eight logits (from expert e0); -inf behind the last expert
__device__ __forceinline__ void load_logits(const uint16_t* row, int e0, int E, float (&v)[8]) {
  Raw8<uint16_t> r;
  fetch8(row, e0, E, E < 8, r);
  if (ragged(E)) settle8(e0, E, r);
  widen8(r, v);
  if (e0 + 8 > E) {
#pragma unroll
    for (int i = 0; i < 8; i++) v[i] = e0 + i < E ? v[i] : -INFINITY;
  }
}

// the softmax of a group's logits: v becomes the probabilities, z the
// log-sum-exp.  False where no logit is above -inf (or one is a NaN).
template <int L>
__device__ __forceinline__ bool group_softmax(float (&v)[8], float& z) {
  float m = v[0];
#pragma unroll
  for (int j = 1; j < 8; j++) m = fmaxf(m, v[j]);
  m = group_max<L>(m);
  float s = 0.f;
#pragma unroll
  for (int j = 0; j < 8; j++) {
    v[j] = __builtin_amdgcn_exp2f((v[j] - m) * kLog2e);
    s += v[j];
  }
  s = group_sum<L>(s);
  const float r = 1.0f / s;
#pragma unroll
  for (int j = 0; j < 8; j++) v[j] *= r;
  z = fmaf(__builtin_amdgcn_logf(s), kLn2, m);
  return m > -INFINITY;
}

__device__ __forceinline__ int clamped(int v, int T) { return min(max(v, 0), T); }

// the last sequence that starts at or before token t (-1: none)
__device__ __forceinline__ int sequence_of(const int32_t* seq, int S, int t) {
  int lo = 0, hi = S;  // the first of [0, S) that starts behind t
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (seq[mid] <= t)
      lo = mid + 1;
    else
      hi = mid;
  }
  return lo - 1;
}

// Workspace of a balance call: a workgroup's chunk of tokens is cut at the
// sequences' borders into pieces; piece (chunk c, sequence s) has the slot
// c + s (distinct, since both only rise along the tokens).
struct BalanceLayout {
  int chunk, chunks, slots;
  size_t p, c, zn, part, total;  // byte offsets
};
__host__ __device__ inline BalanceLayout balance_layout(int T, int E, int S) {
  BalanceLayout b;
  const int per = (T + 1023) / 1024;
  b.chunk = per > 64 ? per : 64;
  b.chunks = T > 0 ? (T + b.chunk - 1) / b.chunk : 0;
  b.slots = b.chunks + S;
  const size_t cell = (size_t)b.slots * E * 4;
  b.p = 0;
  b.c = b.p + cell;
  b.zn = b.c + cell;
  b.part = b.zn + (size_t)b.slots * 8;
  b.total = b.part + (size_t)S * ((E + 15) / 16) * 4 + (size_t)S * 8;
  return b;
}

template <int L>
__global__ __launch_bounds__(kThreads) void balance_pieces_kernel(const uint16_t* __restrict__ logits,
                                                                  const int32_t* __restrict__ ids, int T, int E, int k,
                                                                  const int32_t* __restrict__ seq, int S, int chunk,
                                                                  float* __restrict__ part_p,
                                                                  int32_t* __restrict__ part_c,
                                                                  float2* __restrict__ part_zn) {
  constexpr int kGroups = kThreads / L;
  __shared__ int hist[L * 8];
  __shared__ float red[kThreads / 64][L * 8];
  __shared__ float redz[kThreads / 64];
  __shared__ int redn[kThreads / 64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int j = threadIdx.x % L, group = threadIdx.x / L;
  const int e0 = j * 8;
  const int c0 = blockIdx.x * chunk, c1 = min(c0 + chunk, T);
  int s = seq ? max(sequence_of(seq, S, c0), 0) : 0;
  for (; s < S; s++) {
    const int a = seq ? max(seq[s], c0) : c0;
    if (a >= c1) break;
    const int b = seq ? min(seq[s + 1], c1) : c1;
    if (b <= a) continue;
    for (int e = threadIdx.x; e < E; e += kThreads) hist[e] = 0;
    __syncthreads();
    float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    float z2 = 0.f;
    int n = 0;
    for (int t = a + group; t < b; t += kGroups) {
      float v[8], z;
      load_logits(logits + (size_t)t * E, e0, E, v);
      bool valid = false;
      for (int q = j; q < k; q += L) valid |= (unsigned)ids[(size_t)t * k + q] < (unsigned)E;
      const bool some = group_any<L>(valid);
      const bool live = group_softmax<L>(v, z) && some;
      if (live) {
        for (int q = j; q < k; q += L) {
          const int id = ids[(size_t)t * k + q];
          if ((unsigned)id < (unsigned)E) atomicAdd(&hist[id], 1);
        }
#pragma unroll
        for (int i = 0; i < 8; i++) acc[i] += v[i];
        z2 = fmaf(z, z, z2);
        n++;
      }
    }
    // the wave's groups, then the waves, in order
#pragma unroll
    for (int o = L; o < 64; o <<= 1) {
#pragma unroll
      for (int i = 0; i < 8; i++) acc[i] += __shfl_xor(acc[i], o, 64);
      z2 += __shfl_xor(z2, o, 64);
      n += __shfl_xor(n, o, 64);
    }
    if (lane < L) {
#pragma unroll
      for (int i = 0; i < 8; i++) red[wave][e0 + i] = acc[i];
    }
    if (lane == 0) redz[wave] = z2, redn[wave] = n;
    __syncthreads();
    const size_t slot = (size_t)blockIdx.x + s;
    for (int e = threadIdx.x; e < E; e += kThreads) {
      float v = red[0][e];
#pragma unroll
      for (int w = 1; w < kThreads / 64; w++) v += red[w][e];
      part_p[slot * E + e] = v;
      part_c[slot * E + e] = hist[e];
    }
    if (threadIdx.x == 0) {
      float zz = redz[0];
      int nn = redn[0];
#pragma unroll
      for (int w = 1; w < kThreads / 64; w++) zz += redz[w], nn += redn[w];
      part_zn[slot] = make_float2(zz, __int_as_float(nn));
    }
    __syncthreads();
  }
}

// One sequence's pieces: 16 experts x 64 piece groups per workgroup.
constexpr int kSumThreads = 1024;
constexpr int kSumCols = 16;
__global__ __launch_bounds__(kSumThreads) void balance_sequences_kernel(
    const float* __restrict__ part_p, const int32_t* __restrict__ part_c, const float2* __restrict__ part_zn, int T,
    int E, const int32_t* __restrict__ seq, int chunk, int32_t* __restrict__ counts, int32_t* __restrict__ tokens,
    float* __restrict__ part, float* __restrict__ seq_z) {
  constexpr int kRows = kSumThreads / kSumCols;
  __shared__ float redp[kRows][kSumCols + 1];
  __shared__ int redc[kRows][kSumCols + 1];
  const int s = blockIdx.x;
  const int col = threadIdx.x % kSumCols, row = threadIdx.x / kSumCols;
  const int e = blockIdx.y * kSumCols + col;
  const int a = seq ? clamped(seq[s], T) : 0, b = seq ? clamped(seq[s + 1], T) : T;
  float p = 0.f;
  int c = 0;
  const int first = b > a ? a / chunk : 0, last = b > a ? (b - 1) / chunk : -1;
  if (e < E) {
    for (int i = first + row; i <= last; i += kRows) {
      const size_t slot = (size_t)i + s;
      p += part_p[slot * E + e];
      c += part_c[slot * E + e];
    }
  }
  redp[row][col] = p;
  redc[row][col] = c;
  __syncthreads();
  if (threadIdx.x < 64) {  // wave 0: columns, then the sum of c * p over them
    float cp = 0.f;
    if (threadIdx.x < kSumCols && e < E) {
      p = 0.f;
      c = 0;
      for (int i = 0; i < kRows; i++) p += redp[i][col], c += redc[i][col];
      counts[(size_t)s * E + e] = c;
      cp = (float)c * p;
    }
    cp = wave_sum(cp);
    if (threadIdx.x == 0) part[(size_t)s * gridDim.y + blockIdx.y] = cp;
  } else if (blockIdx.y == 0 && threadIdx.x < 128) {  // wave 1: tokens and z
    float z = 0.f;
    int n = 0;
    for (int i = first + (int)threadIdx.x - 64; i <= last; i += 64) {
      const float2 zn = part_zn[(size_t)i + s];
      z += zn.x;
      n += __float_as_int(zn.y);
    }
    z = wave_sum(z);
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) n += __shfl_xor(n, o, 64);
    if (threadIdx.x == 64) {
      seq_z[s] = z;
      tokens[s] = n;
    }
  }
}

__global__ __launch_bounds__(kThreads) void balance_losses_kernel(const float* __restrict__ part,
                                                                  const float* __restrict__ seq_z, int E, int k, int S,
                                                                  int blocks, int32_t* __restrict__ tokens,
                                                                  float* __restrict__ losses) {
  __shared__ float redb[kThreads / 64], redz[kThreads / 64];
  __shared__ int redn[kThreads / 64], redu[kThreads / 64];
  float loss = 0.f, z = 0.f;
  int n = 0, used = 0;
  for (int s = threadIdx.x; s < S; s += kThreads) {
    const int ns = tokens[s];
    if (ns > 0) {
      float cp = 0.f;
      for (int i = 0; i < blocks; i++) cp += part[(size_t)s * blocks + i];
      loss += cp * ((float)E / (float)k) / ((float)ns * (float)ns);
      z += seq_z[s];
      n += ns;
      used++;
    }
  }
  loss = wave_sum(loss);
  z = wave_sum(z);
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) n += __shfl_xor(n, o, 64), used += __shfl_xor(used, o, 64);
  if ((threadIdx.x & 63) == 0) {
    const int w = threadIdx.x >> 6;
    redb[w] = loss, redz[w] = z, redn[w] = n, redu[w] = used;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
#pragma unroll
    for (int w = 1; w < kThreads / 64; w++) loss += redb[w], z += redz[w], n += redn[w], used += redu[w];
    tokens[S] = n;
    tokens[S + 1] = used;
    losses[0] = used > 0 ? loss / (float)used : 0.f;
    losses[1] = n > 0 ? z / (float)n : 0.f;
  }
}

// dlogits.  LOSSES: the balance and z losses' part (else the gates' alone, and
// logits, seq, counts and tokens are not read).
template <int L, typename O, bool LOSSES>
__global__ __launch_bounds__(kThreads) void route_backward_kernel(
    const uint16_t* __restrict__ logits, const int32_t* __restrict__ ids, const float* __restrict__ gates,
    const float* __restrict__ dgates, int T, int E, int k, const int32_t* __restrict__ seq, int S,
    const int32_t* __restrict__ counts, const int32_t* __restrict__ tokens, const float* __restrict__ dlosses,
    int chunk, O* __restrict__ dlogits) {
  constexpr int kGroups = kThreads / L;
  const int j = threadIdx.x % L, group = threadIdx.x / L;
  const int e0 = j * 8;
  const int c0 = blockIdx.x * chunk, c1 = min(c0 + chunk, T);
  float da = 0.f, b = 0.f;
  int s = 0, s_end = T, s_have = -1;
  float c[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if constexpr (LOSSES) {
    da = dlosses[0] * (float)E / ((float)k * (float)max(tokens[S + 1], 1));
    b = 2.f * dlosses[1] / (float)max(tokens[S], 1);
    if (seq) {
      s = sequence_of(seq, S, c0);
      s_end = s + 1 <= S ? seq[s + 1] : T;
    }
  }
  for (int t = c0 + group; t < c1; t += kGroups) {
    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}, z = 0.f;
    bool live = true;
    if constexpr (LOSSES) {
      load_logits(logits + (size_t)t * E, e0, E, v);
      while (seq && t >= s_end && s < S) {
        s++;
        s_end = s < S ? seq[s + 1] : T;
      }
      live = s >= 0 && s < S;
    }
    // the slots: lane j takes the slots j, j + L, ...
    bool valid = false;
    float qd = 0.f;
    for (int q = j; q < k; q += L) {
      const size_t r = (size_t)t * k + q;
      const bool ok = (unsigned)ids[r] < (unsigned)E;
      valid |= ok;
      if (dgates) {
        const float g = ok ? gates[r] : 0.f;
        if (g != 0.f) qd = fmaf(g, dgates[r], qd);
      }
    }
    live = group_any<L>(valid) && live;
    if constexpr (LOSSES) {
      live = group_softmax<L>(v, z) && live;
      float pc = 0.f;
      if (live) {
        if (s != s_have) {
          float sum = 0.f;
#pragma unroll
          for (int i = 0; i < 8; i++) {
            c[i] = e0 + i < E ? (float)counts[(size_t)s * E + e0 + i] : 0.f;
            sum += c[i];
          }
          sum = group_sum<L>(sum);
          const float n = (float)max(tokens[s], 1);
          const float a = da / (n * n), mean = sum / (float)E;
#pragma unroll
          for (int i = 0; i < 8; i++) c[i] = (c[i] - mean) * a;
          s_have = s;
        }
#pragma unroll
        for (int i = 0; i < 8; i++) pc = fmaf(v[i], c[i], pc);
      }
      pc = group_sum<L>(pc);
      const float bz = b == 0.f ? 0.f : b * z;
#pragma unroll
      for (int i = 0; i < 8; i++) v[i] = live ? v[i] * (c[i] - pc + bz) : 0.f;
    }
    if (dgates) {
      qd = group_sum<L>(qd);
      for (int q0 = 0; q0 < k; q0 += L) {
        int id = -1;
        float d = 0.f;
        if (q0 + j < k) {
          const size_t r = (size_t)t * k + q0 + j;
          id = ids[r];
          const float g = (unsigned)id < (unsigned)E ? gates[r] : 0.f;
          if (g != 0.f) d = g * (dgates[r] - qd);
        }
        const int m = min(L, k - q0);
        for (int q = 0; q < m; q++) {
          const int src = ((threadIdx.x & 63) & ~(L - 1)) + q;
          const int at = __shfl(id, src, 64) - e0;
          const float dq = __shfl(d, src, 64);
#pragma unroll
          for (int i = 0; i < 8; i++) v[i] += at == i && live ? dq : 0.f;
        }
      }
    }
    store8(dlogits + (size_t)t * E, e0, E, v);
  }
}

// f(the lanes of a token's group as a constant)
template <typename F>
void with_lanes(int E, F f) {
  const int pieces = (E + 7) / 8;
  if (pieces <= 1)
    f(std::integral_constant<int, 1>{});
  else if (pieces <= 2)
    f(std::integral_constant<int, 2>{});
  else if (pieces <= 4)
    f(std::integral_constant<int, 4>{});
  else if (pieces <= 8)
    f(std::integral_constant<int, 8>{});
  else if (pieces <= 16)
    f(std::integral_constant<int, 16>{});
  else if (pieces <= 32)
    f(std::integral_constant<int, 32>{});
  else
    f(std::integral_constant<int, 64>{});
}

}  // namespace

size_t balance_workspace_bytes(int T, int E, int S) { return balance_layout(T, E, S).total; }

hipError_t launch_balance(const uint16_t* logits, const int32_t* ids, int T, int E, int k, const int32_t* seq, int S,
                          int32_t* counts, int32_t* tokens, float* losses, void* workspace, hipStream_t stream) {
  const BalanceLayout b = balance_layout(T, E, S);
  char* ws = static_cast<char*>(workspace);
  float* part_p = reinterpret_cast<float*>(ws + b.p);
  int32_t* part_c = reinterpret_cast<int32_t*>(ws + b.c);
  float2* part_zn = reinterpret_cast<float2*>(ws + b.zn);
  const int blocks = (E + kSumCols - 1) / kSumCols;
  float* part = reinterpret_cast<float*>(ws + b.part);
  float* seq_z = part + (size_t)S * blocks;
  hipError_t e = hipSuccess;
  if (b.chunks > 0) {
    with_lanes(E, [&](auto lanes) {
      hipLaunchKernelGGL((balance_pieces_kernel<decltype(lanes)::value>), dim3(b.chunks), dim3(kThreads), 0, stream,
                         logits, ids, T, E, k, seq, S, b.chunk, part_p, part_c, part_zn);
    });
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(balance_sequences_kernel, dim3(S, blocks), dim3(kSumThreads), 0, stream, part_p, part_c, part_zn,
                     T, E, seq, b.chunk, counts, tokens, part, seq_z);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(balance_losses_kernel, dim3(1), dim3(kThreads), 0, stream, part, seq_z, E, k, S, blocks, tokens,
                     losses);
  return hipGetLastError();
}

hipError_t launch_route_backward(const uint16_t* logits, const int32_t* ids, const float* gates, const float* dgates,
                                 int T, int E, int k, const int32_t* seq, int S, const int32_t* counts,
                                 const int32_t* tokens, const float* dlosses, void* dlogits, bool dlogits_f32,
                                 hipStream_t stream) {
  const int chunk = 64, chunks = (T + chunk - 1) / chunk;
  with_lanes(E, [&](auto lanes) {
    constexpr int L = decltype(lanes)::value;
    auto with_out = [&](auto elem) {
      using O = decltype(elem);
      if (dlosses)
        hipLaunchKernelGGL((route_backward_kernel<L, O, true>), dim3(chunks), dim3(kThreads), 0, stream, logits, ids,
                           gates, dgates, T, E, k, seq, S, counts, tokens, dlosses, chunk, static_cast<O*>(dlogits));
      else
        hipLaunchKernelGGL((route_backward_kernel<L, O, false>), dim3(chunks), dim3(kThreads), 0, stream, logits, ids,
                           gates, dgates, T, E, k, seq, S, counts, tokens, dlosses, chunk, static_cast<O*>(dlogits));
    };
    if (dlogits_f32)
      with_out(float{});
    else
      with_out(uint16_t{});
  });
  return hipGetLastError();
}

}  // namespace mxfp4
