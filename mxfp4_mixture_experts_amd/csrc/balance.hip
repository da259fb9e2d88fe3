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
// and a token's maximum and sums take log2(L) register moves.  A group fetches
// its next token's logits and slots before it works on this one's.

#include <type_traits>

#include "kernels.h"
#include "rows.h"

namespace mxfp4 {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// the number of a thread's group: the same for a whole wave where L is 64, so
// that a token's addresses are scalar there
template <int L>
__device__ __forceinline__ int group_of_thread() {
  return L == 64 ? __builtin_amdgcn_readfirstlane(threadIdx.x / L) : (int)threadIdx.x / L;
}
template <int L>
__device__ __forceinline__ bool group_any(bool p) {
  const uint64_t m = __ballot(p);
  if constexpr (L == 64) return m != 0;
  const int base = (threadIdx.x & 63) & ~(L - 1);
  return ((m >> base) & ((1ull << (L & 63)) - 1)) != 0;
}

// A lane's eight logits (from expert e0) of a token's row; -inf behind the last
// expert.  Every lane loads eight that the row has, whatever part of them is its
// own: settle_logits sorts that out, where E is not 8 L.
template <int L>
__device__ __forceinline__ void fetch_logits(const uint16_t* row, int e0, int E, Raw8<uint16_t>& r) {
  if (L == 1 && E < 8)
    fetch8(row, e0, E, true, r);
  else
    fetch8_full(row + min(e0, E - 8), r);
}
template <int L>
__device__ __forceinline__ void settle_logits(Raw8<uint16_t> r, int e0, int E, float (&v)[8]) {
  if (E != 8 * L && E > 8) settle8(e0, E, r);
  widen8(r, v);
  if (E != 8 * L) {
#pragma unroll
    for (int i = 0; i < 8; i++) v[i] = e0 + i < E ? v[i] : -INFINITY;
  }
}

// a lane's eight counts of a sequence's row; 0 behind the last expert
template <int L>
__device__ __forceinline__ void load_counts(const int32_t* row, int e0, int E, int (&c)[8]) {
  const float* words = reinterpret_cast<const float*>(row);  // moved as they are
  Raw8<float> r = {};
  if (L == 1 && E < 8) {
    fetch8(words, e0, E, true, r);
  } else if (e0 < E) {
    fetch8_full(words + min(e0, E - 8), r);
    settle8(e0, E, r);
  }
#pragma unroll
  for (int i = 0; i < 4; i++) c[i] = __float_as_int(r.a[i]), c[4 + i] = __float_as_int(r.b[i]);
}

// The exponentials of a group's logits against a common m, in place; m is -inf
// where no logit is above that.  While every token of the wave has its largest
// logit in [-kNear, kNear], m is 0 and no maximum over the lanes is needed: no
// exponential passes fp32's range, and a sum of them is at least e^-16, so that
// the only probabilities which vanish with their exponentials lie under e^-71.
// (Router logits lie there.  65536 x 512: balance 22.5 us, gradient 31.6; with the
// maxima looked for 24.4 and 32.3.  A wider range is quicker for larger logits, but
// the product's rounding grows with them: 2^-20 of p at 16, 2^-18 at 64.)  Otherwise
// the maxima are looked for, and m is 0 still for a token whose own lies there --
// the same bits whatever the tokens beside it in the wave hold -- and the row's
// maximum for another, taken off before the product with log2 e: rounded apart,
// m log2 e would be off by far more than an exponent's range where m is large.
constexpr float kNear = 16.f;
template <int L>
__device__ __forceinline__ void group_exp(float (&v)[8], float& m) {
  float top = v[0];
#pragma unroll
  for (int j = 1; j < 8; j++) top = fmaxf(top, v[j]);
  const bool near = group_any<L>(top >= -kNear) && top <= kNear;
  if (__ballot(!near) == 0) {
    m = 0.f;
#pragma unroll
    for (int j = 0; j < 8; j++) v[j] = __builtin_amdgcn_exp2f(v[j] * kLog2e);
    return;
  }
  m = group_max<L>(top);
  if (m >= -kNear && m <= kNear) m = 0.f;
  const float off = m > -INFINITY ? m : 0.f;
#pragma unroll
  for (int j = 0; j < 8; j++) v[j] = __builtin_amdgcn_exp2f((v[j] - off) * kLog2e);
}

// The sums of three values over a group.  A whole wave adds them together: after
// each exchange across rows a row holds the partial sums of one of them.
template <int L>
__device__ __forceinline__ void group_sum3(float& a, float& b, float& c) {
  if constexpr (L == 64) {
    const auto ab = __builtin_amdgcn_permlane32_swap(bits(a), bits(b), false, false);
    const auto cc = __builtin_amdgcn_permlane32_swap(bits(c), bits(c), false, false);
    const float x = __uint_as_float(ab[0]) + __uint_as_float(ab[1]);  // a in rows 0, 1; b in rows 2, 3
    const float y = __uint_as_float(cc[0]) + __uint_as_float(cc[1]);
    const auto xy = __builtin_amdgcn_permlane16_swap(bits(x), bits(y), false, false);
    const float rows = group_sum<16>(__uint_as_float(xy[0]) + __uint_as_float(xy[1]));  // a, c, b, c
    a = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(rows), 0));
    b = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(rows), 32));
    c = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(rows), 16));
  } else {
    a = group_sum<L>(a);
    b = group_sum<L>(b);
    c = group_sum<L>(c);
  }
}

// the log-sum-exp from m and the sum of the exponentials
__device__ __forceinline__ float log_sum(float m, float sum) {
  return fmaf(__builtin_amdgcn_logf(sum), kLn2, m);
}

__device__ __forceinline__ int clamped(int v, int T) { return min(max(v, 0), T); }

// The last sequence that starts at or before token t (-1: none).  A whole wave
// looks for it, 64 starts at a time: one load's latency up to 64 sequences.
// Whatever seq holds, the result lies in [-1, S).
__device__ __forceinline__ int sequence_of(const int32_t* seq, int S, int t) {
  const int lane = threadIdx.x & 63;
  int lo = -1, hi = S;  // starts up to lo lie at or before t; those from hi on are not looked at
  while (hi - lo > 1) {
    const int stride = (hi - lo - 1 + 63) / 64;
    const int at = lo + 1 + lane * stride;
    const int n = __popcll(__ballot(at < hi && seq[min(at, hi - 1)] <= t));
    if (n == 0) break;
    lo += 1 + (n - 1) * stride;
    hi = min(lo + stride, hi);
  }
  return lo;
}

// Workspace of a balance call: a workgroup's chunk of tokens is cut at the
// sequences' borders into pieces; piece (chunk c, sequence s) has the slot
// c + s (distinct, since both only rise along the tokens).  A workgroup takes
// its pieces one after another, 1.2 to 2 us each, so chunks are no longer than
// the mean sequence, from 64 tokens (which fill the chip from 16384 tokens on)
// down to 4; beyond 32768 tokens they grow, so that there are never more than
// 512 to add up.  Lengths far from their mean are what this does not serve: one
// sequence of 4032 beside 64 of one token (4096 x 32) takes 86 us, of 64512 beside
// 1024 of one (65536 x 512) 191 us, where 64 of random lengths take 15 and 23 us.
constexpr int kSumCols = 64;  // experts per workgroup of the second launch
struct BalanceLayout {
  int chunk, chunks, slots, blocks;
  size_t zn, p, c, part, arrivals, total;  // byte offsets
};
BalanceLayout balance_layout(int T, int E, int S) {
  BalanceLayout b;
  const int per = (T + 511) / 512, mean = T / S;
  b.chunk = mean > 64 ? 64 : mean > 4 ? mean : 4;
  if (b.chunk < per) b.chunk = per;
  b.chunks = T > 0 ? (T + b.chunk - 1) / b.chunk : 0;
  b.slots = b.chunks + S;
  b.blocks = (E + kSumCols - 1) / kSumCols;
  const size_t cell = (size_t)b.slots * E * 4;
  b.zn = 0;
  b.p = b.zn + (size_t)b.slots * 8;
  b.c = b.p + cell;
  b.part = b.c + cell;
  b.arrivals = b.part + (size_t)S * b.blocks * 4 + (size_t)S * 4;
  b.total = b.arrivals + 4;
  return b;
}

// The threads of a piece's workgroup: more where a wave holds few tokens.
//
// What bounds the first launch: vector instructions (83 a token of 512 experts:
// at four cycles each about 9 of the 18 us for 65536 of them; 67 MB are 13 us at the
// rate of a copy) and the latency of a workgroup's first loads and last sums; for
// 4096 tokens of 32 experts (4 us) these alone.
template <int L>
constexpr int kPieceThreads = L >= 16 ? 1024 : 256;

template <int L>
__global__ __launch_bounds__(kPieceThreads<L>) void balance_pieces_kernel(
    const uint16_t* __restrict__ logits, const int32_t* __restrict__ ids, int T, int E, int k,
    const int32_t* __restrict__ seq, int S, int chunk, float* __restrict__ part_p, int32_t* __restrict__ part_c,
    float2* __restrict__ part_zn, int* __restrict__ arrivals) {
  constexpr int kThreads = kPieceThreads<L>;
  constexpr int kGroups = kThreads / L;
  constexpr int kWaves = kThreads / 64;
  __shared__ int hist[L * 8];
  __shared__ float red[kWaves][L * 8];
  __shared__ float redz[kWaves];
  __shared__ int redn[kWaves];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int j = threadIdx.x % L, group = group_of_thread<L>();
  const int e0 = j * 8;
  const int c0 = blockIdx.x * chunk, c1 = min(c0 + chunk, T);
  if (blockIdx.x == 0 && threadIdx.x == 0) *arrivals = 0;  // for the second launch
  int s = seq ? max(sequence_of(seq, S, c0), 0) : 0;
  while (s < S) {
    const int a = seq ? max(seq[s], c0) : c0;
    if (a >= c1) break;
    const int b = seq ? min(seq[s + 1], c1) : c1;
    if (b <= a) {
      // an empty sequence: on to the last one that starts there, behind however
      // many more (a call with 65535 inside a chunk: 0.20 ms; one after the other 6.5 ms)
      s = max(s + 1, sequence_of(seq, S, a));
      continue;
    }
    Raw8<uint16_t> next;
    int id_next = -1;
    auto fetch = [&](int t) {
      fetch_logits<L>(logits + (size_t)t * E, e0, E, next);
      id_next = j < k ? ids[(size_t)t * k + j] : -1;
    };
    if (a + group < b) fetch(a + group);
    for (int e = threadIdx.x; e < E; e += kThreads) hist[e] = 0;
    __syncthreads();
    float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    float z2 = 0.f;
    int n = 0;
    for (int t = a + group; t < b; t += kGroups) {
      float v[8], m;
      settle_logits<L>(next, e0, E, v);
      const int id = id_next;
      if (t + kGroups < b) fetch(t + kGroups);
      bool valid = (unsigned)id < (unsigned)E;
      if constexpr (L < kMaxTopK)
        for (int q = j + L; q < k; q += L) valid |= (unsigned)ids[(size_t)t * k + q] < (unsigned)E;
      const bool some = group_any<L>(valid);
      group_exp<L>(v, m);
      float sum = v[0];
#pragma unroll
      for (int i = 1; i < 8; i++) sum += v[i];
      sum = group_sum<L>(sum);
      if (some && m > -INFINITY) {
        if ((unsigned)id < (unsigned)E) atomicAdd(&hist[id], 1);
        if constexpr (L < kMaxTopK)
          for (int q = j + L; q < k; q += L) {
            const int at = ids[(size_t)t * k + q];
            if ((unsigned)at < (unsigned)E) atomicAdd(&hist[at], 1);
          }
        const float r = __builtin_amdgcn_rcpf(sum);
        const float z = log_sum(m, sum);
#pragma unroll
        for (int i = 0; i < 8; i++) acc[i] = fmaf(v[i], r, acc[i]);
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
      for (int w = 1; w < kWaves; w++) v += red[w][e];
      part_p[slot * E + e] = v;
      part_c[slot * E + e] = hist[e];
    }
    if (threadIdx.x == 0) {
      float zz = redz[0];
      int nn = redn[0];
#pragma unroll
      for (int w = 1; w < kWaves; w++) zz += redz[w], nn += redn[w];
      part_zn[slot] = make_float2(zz, __int_as_float(nn));
    }
    s++;
    __syncthreads();
  }
}

// One sequence's pieces: 64 experts x 16 piece groups per workgroup, the pieces
// of a group in order (four loads under way), then the groups in order.  Each
// workgroup leaves its share of the losses in the workspace and counts itself
// in; the last one to do so adds the shares in order and writes the losses, so
// the sum does not depend on which that is.  The shares go through
// device-scope stores and loads (sc1: past the XCD's own L2 to the level that
// all share), and a workgroup counts itself in once its stores are complete
// (vmcnt); a release and acquire instead write back and drop whole L2s, 4 us for
// one workgroup and 9 us for 296.  arrivals == NULL: no counting, a third launch
// adds the shares.
constexpr int kSumThreads = 1024;
constexpr int kSumDepth = 4;

template <typename V>
__device__ __forceinline__ V load_shared(const V* p) {  // written by another workgroup of this launch
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
template <typename V>
__device__ __forceinline__ void store_shared(V* p, V v) {
  __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// The losses and the tokens' totals from the shares of every sequence and block
// of experts, by one workgroup in a fixed order.
__device__ __forceinline__ void sum_losses(const float* part, const float* seq_z, int S, int blocks, int32_t* tokens,
                                           float* losses, float* redf, int* redi) {
  constexpr int kWaves = kSumThreads / 64;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  float loss = 0.f, z = 0.f;
  int n = 0, used = 0;
  for (int i = threadIdx.x; i < S * blocks; i += kSumThreads) loss += load_shared(part + i);
  for (int i = threadIdx.x; i < S; i += kSumThreads) {
    const int ns = load_shared(tokens + i);
    z += load_shared(seq_z + i);
    n += ns;
    used += ns > 0;
  }
  loss = group_sum<64>(loss);
  z = group_sum<64>(z);
  n = group_sum<64>(n);
  used = group_sum<64>(used);
  if (lane == 0) {
    redf[wave] = loss, redf[kWaves + wave] = z;
    redi[wave] = n, redi[kWaves + wave] = used;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
#pragma unroll
    for (int w = 1; w < kWaves; w++)
      loss += redf[w], z += redf[kWaves + w], n += redi[w], used += redi[kWaves + w];
    tokens[S] = n;
    tokens[S + 1] = used;
    losses[0] = used > 0 ? loss / (float)used : 0.f;
    losses[1] = n > 0 ? z / (float)n : 0.f;
  }
}

__global__ __launch_bounds__(kSumThreads) void balance_sequences_kernel(
    const float* __restrict__ part_p, const int32_t* __restrict__ part_c, const float2* __restrict__ part_zn, int T,
    int E, int k, const int32_t* __restrict__ seq, int S, int chunk, int32_t* __restrict__ counts, int32_t* tokens,
    float* __restrict__ losses, float* part, float* seq_z, int* arrivals) {
  constexpr int kRows = kSumThreads / kSumCols;
  __shared__ float redp[kRows][kSumCols];
  __shared__ int redc[kRows][kSumCols];
  __shared__ float z_all;
  __shared__ int n_all, last_all;
  const int s = blockIdx.x;
  const int col = threadIdx.x % kSumCols, row = threadIdx.x / kSumCols;  // a wave is one row
  const int e = blockIdx.y * kSumCols + col;
  const int a = seq ? clamped(seq[s], T) : 0, b = seq ? clamped(seq[s + 1], T) : T;
  const int first = b > a ? a / chunk : 0, last = b > a ? (b - 1) / chunk : -1;
  float p = 0.f, z = 0.f;
  int c = 0, n = 0;
  if (e < E) {
    for (int i = first + row; i <= last; i += kRows * kSumDepth) {
      float pv[kSumDepth];
      int cv[kSumDepth];
#pragma unroll
      for (int u = 0; u < kSumDepth; u++) {
        const size_t slot = (size_t)min(i + u * kRows, last) + s;
        pv[u] = part_p[slot * E + e];
        cv[u] = part_c[slot * E + e];
      }
#pragma unroll
      for (int u = 0; u < kSumDepth; u++) {
        const bool in = i + u * kRows <= last;
        p += in ? pv[u] : 0.f;
        c += in ? cv[u] : 0;
      }
    }
  }
  if (row == 1) {  // wave 1 adds the tokens and z^2 beside
    for (int i = first + col; i <= last; i += 64) {
      const float2 zn = part_zn[(size_t)i + s];
      z += zn.x;
      n += __float_as_int(zn.y);
    }
    z = group_sum<64>(z);
    n = group_sum<64>(n);
    if (col == 0) z_all = z, n_all = n;
  }
  redp[row][col] = p;
  redc[row][col] = c;
  __syncthreads();
  if (row == 0) {
#pragma unroll
    for (int i = 1; i < kRows; i++) p += redp[i][col], c += redc[i][col];
    if (e < E) counts[(size_t)s * E + e] = c;
    const float cp = group_sum<64>((float)c * p);
    const bool alone = gridDim.x == 1 && gridDim.y == 1;
    if (col == 0 && alone) {
      n = n_all;
      tokens[0] = tokens[1] = n;
      tokens[2] = n > 0;
      losses[0] = n > 0 ? cp * ((float)E / (float)k) / ((float)n * (float)n) : 0.f;
      losses[1] = n > 0 ? z_all / (float)n : 0.f;
      last_all = 0;
    } else if (col == 0) {
      n = n_all;
      store_shared(part + (size_t)s * gridDim.y + blockIdx.y,
                   n > 0 ? cp * ((float)E / (float)k) / ((float)n * (float)n) : 0.f);
      if (blockIdx.y == 0) {
        store_shared(seq_z + s, z_all);
        store_shared(tokens + s, n);
      }
      last_all = 0;
      if (arrivals) {
        asm volatile("" ::: "memory");
        __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0)
        asm volatile("" ::: "memory");
        last_all = __hip_atomic_fetch_add(arrivals, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) ==
                   (int)(gridDim.x * gridDim.y) - 1;
      }
    }
  }
  __syncthreads();
  if (last_all) sum_losses(part, seq_z, S, gridDim.y, tokens, losses, redp[0], redc[0]);
}

__global__ __launch_bounds__(kSumThreads) void balance_losses_kernel(const float* part, const float* seq_z, int S,
                                                                     int blocks, int32_t* tokens, float* losses) {
  __shared__ float redf[2 * kSumThreads / 64];
  __shared__ int redi[2 * kSumThreads / 64];
  sum_losses(part, seq_z, S, blocks, tokens, losses, redf, redi);
}

constexpr int kRouteThreads = 256;
// Tokens of a workgroup: one or more for each group, eight where a token takes
// half a wave or a whole one (65536 tokens of 512 experts then fill every wave
// slot of the chip; 16 each: 46 us against 37).
template <int L>
constexpr int kRouteChunk = L >= 32 ? 8 * kRouteThreads / L : kRouteThreads / L > 64 ? kRouteThreads / L : 64;

// dlogits.  LOSSES: the balance and z losses' part (else the gates' alone, and
// logits, seq, counts and tokens are not read).
//
// The slots' values meet their experts' lanes through a wave's own LDS row: one
// write and one read a token, where comparing every slot with every lane's eight
// experts takes 3 x 8 k vector instructions.  A token's slots normally hold
// distinct experts; the lowest slot of a repeated one goes first, the others in
// further rounds, so the order of their sum is fixed.  (Comparing: 89 us for
// 65536 tokens of 512 experts with 8 slots; this way 46.)
//
// What bounds it: 181 vector instructions a token of 512 experts, at four cycles
// each about 19 of the 31 us for 65536 of them, where 141 MB are 26 us at the rate of
// a copy.  The gates' part alone (65536 x 512 x 8, bf16 out) takes 14.8 us, 5.0 TB/s.
template <int L, typename O, bool LOSSES>
__global__ __launch_bounds__(kRouteThreads, L == 64 ? 8 : 1) void route_backward_kernel(
    const uint16_t* __restrict__ logits, const int32_t* __restrict__ ids, const float* __restrict__ gates,
    const float* __restrict__ dgates, int T, int E, int k, const int32_t* __restrict__ seq, int S,
    const int32_t* __restrict__ counts, const int32_t* __restrict__ tokens, const float* __restrict__ dlosses,
    int chunk, O* __restrict__ dlogits) {
  constexpr int kGroups = kRouteThreads / L;
  constexpr int kNone = 0x7fffffff;
  __shared__ __align__(16) float slot_value[kRouteThreads * 8];
  __shared__ __align__(16) int slot_owner[kRouteThreads * 8];
  const int j = threadIdx.x % L, group = group_of_thread<L>();
  const int e0 = j * 8;
  float* value = slot_value + group * (L * 8);  // a group's experts; other groups never touch them
  int* owner = slot_owner + group * (L * 8);
#pragma unroll
  for (int i = 0; i < 8; i++) value[e0 + i] = 0.f, owner[e0 + i] = kNone;
  const int c0 = blockIdx.x * chunk, c1 = min(c0 + chunk, T);
  Raw8<uint16_t> l_next;
  int id_next = -1;
  float g_next = 0.f, dg_next = 0.f;
  auto fetch = [&](int t) {
    if constexpr (LOSSES) fetch_logits<L>(logits + (size_t)t * E, e0, E, l_next);
    if (j < k) {
      const size_t r = (size_t)t * k + j;
      id_next = ids[r];
      if (dgates) g_next = gates[r], dg_next = dgates[r];
    }
  };
  if (c0 + group < c1) fetch(c0 + group);
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
    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    const int id = id_next;
    const bool ok = j < k && (unsigned)id < (unsigned)E;
    const float g = ok ? g_next : 0.f;
    const float dg = g != 0.f ? dg_next : 0.f;
    bool live = true;
    if constexpr (LOSSES) {
      settle_logits<L>(l_next, e0, E, v);
      for (int steps = 0; seq && t >= s_end && s < S; steps++) {
        if (steps < 4) {
          s++;
        } else {
          // the first sequence that ends beyond t, by halving, since any number of
          // empty ones may lie between (65535: 11 us for the call; one after the
          // other 6.1 ms).  Up to four borders are quicker passed one by one
          // (halving from the second: 5.6 us for 5540 x 38 in 11 sequences, so 5.5).
          int lo = s, hi = S;
          while (hi - lo > 1) {
            const int mid = (lo + hi) / 2;
            (seq[mid + 1] <= t ? lo : hi) = mid;
          }
          s = hi;
        }
        s_end = s < S ? seq[s + 1] : T;
      }
      live = s >= 0 && s < S;
    }
    if (t + kGroups < c1) fetch(t + kGroups);
    // lane j takes the slots j, j + L, ...; one each where k <= L
    bool valid = ok;
    float qd = g * dg;
    if constexpr (L < kMaxTopK) {
      for (int q = j + L; q < k; q += L) {
        const size_t r = (size_t)t * k + q;
        const bool okq = (unsigned)ids[r] < (unsigned)E;
        valid |= okq;
        if (dgates) {
          const float gq = okq ? gates[r] : 0.f;
          if (gq != 0.f) qd = fmaf(gq, dgates[r], qd);
        }
      }
    }
    live = group_any<L>(valid) && live;
    if constexpr (LOSSES) {
      float m;
      group_exp<L>(v, m);
      live = m > -INFINITY && live;
      if (live && s != s_have) {
        float sum = 0.f;
        int cv[8];
        load_counts<L>(counts + (size_t)s * E, e0, E, cv);
#pragma unroll
        for (int i = 0; i < 8; i++) {
          c[i] = (float)cv[i];
          sum += c[i];
        }
        sum = group_sum<L>(sum);
        const float n = (float)max(tokens[s], 1);
        const float a = da / (n * n), mean = sum / (float)E;
#pragma unroll
        for (int i = 0; i < 8; i++) c[i] = (c[i] - mean) * a;
        s_have = s;
      }
      float sum = 0.f, pc = 0.f;
#pragma unroll
      for (int i = 0; i < 8; i++) {
        sum += v[i];
        pc = fmaf(v[i], c[i], pc);
      }
      group_sum3<L>(sum, pc, qd);
      const float r = __builtin_amdgcn_rcpf(sum);
      const float bz = ((b == 0.f ? 0.f : b * log_sum(m, sum)) - pc * r) * r;
      if (L == 64 ? __ballot(!live) == 0 : true) {
#pragma unroll
        for (int i = 0; i < 8; i++) v[i] = L == 64 || live ? v[i] * fmaf(c[i], r, bz) : 0.f;
      } else {
#pragma unroll
        for (int i = 0; i < 8; i++) v[i] = 0.f;
      }
    } else {
      qd = group_sum<L>(qd);
    }
    if (dgates) {
      for (int q0 = 0; q0 < (L < kMaxTopK ? k : 1); q0 += L) {
        int at = id;
        float d = g != 0.f ? g * (dg - qd) : 0.f;
        bool pending = ok && live;
        if (q0 > 0) {
          pending = false;
          if (q0 + j < k) {
            const size_t r = (size_t)t * k + q0 + j;
            at = ids[r];
            pending = live && (unsigned)at < (unsigned)E;
            const float gq = pending ? gates[r] : 0.f;
            d = gq != 0.f ? gq * (dgates[r] - qd) : 0.f;
          }
        }
        while (__ballot(pending)) {
          if (pending) atomicMin(&owner[at], q0 + j);
          __builtin_amdgcn_wave_barrier();  // a wave's LDS accesses complete in order
          if (pending && owner[at] == q0 + j) {
            value[at] += d;  // one lane per address
            owner[at] = kNone;
            pending = false;
          }
          __builtin_amdgcn_wave_barrier();
        }
      }
      const f32x4_t lo = *reinterpret_cast<const f32x4_t*>(value + e0);
      const f32x4_t hi = *reinterpret_cast<const f32x4_t*>(value + e0 + 4);
      __builtin_amdgcn_wave_barrier();
      *reinterpret_cast<f32x4_t*>(value + e0) = f32x4_t{0.f, 0.f, 0.f, 0.f};
      *reinterpret_cast<f32x4_t*>(value + e0 + 4) = f32x4_t{0.f, 0.f, 0.f, 0.f};
      __builtin_amdgcn_wave_barrier();
#pragma unroll
      for (int i = 0; i < 4; i++) v[i] += lo[i], v[4 + i] += hi[i];
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

constexpr int kArrivals = 128;  // workgroups of the second launch that count themselves in

size_t balance_workspace_bytes(int T, int E, int S) { return balance_layout(T, E, S).total; }

hipError_t launch_balance(const uint16_t* logits, const int32_t* ids, int T, int E, int k, const int32_t* seq, int S,
                          int32_t* counts, int32_t* tokens, float* losses, void* workspace, hipStream_t stream) {
  const BalanceLayout b = balance_layout(T, E, S);
  char* ws = static_cast<char*>(workspace);
  float* part_p = reinterpret_cast<float*>(ws + b.p);
  int32_t* part_c = reinterpret_cast<int32_t*>(ws + b.c);
  float2* part_zn = reinterpret_cast<float2*>(ws + b.zn);
  float* part = reinterpret_cast<float*>(ws + b.part);
  float* seq_z = part + (size_t)S * b.blocks;
  int* arrivals = reinterpret_cast<int*>(ws + b.arrivals);
  const dim3 grid(b.chunks > 0 ? b.chunks : 1);  // without tokens: the arrivals alone
  with_lanes(E, [&](auto lanes) {
    constexpr int L = decltype(lanes)::value;
    hipLaunchKernelGGL((balance_pieces_kernel<L>), grid, dim3(kPieceThreads<L>), 0, stream, logits, ids, T, E, k, seq,
                       S, b.chunk, part_p, part_c, part_zn, arrivals);
  });
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  // Many workgroups wait on each other's arrivals for longer than a launch
  // takes.  By workgroups, with arrivals and with a third launch: 4096 x 32, 8: 10.8
  // and 11.2 us, 64: 14.8 and 14.9, 128: 15.3 and 15.1, 192: 15.3 and 14.0, 512: 18.0 and
  // 14.1; 65536 x 512, 64: 23.1 and 24.4, 128: 22.1 and 22.5, 192: 23.2 and 22.0, 512:
  // 27.1 and 23.1.
  const bool counted = (long long)S * b.blocks <= kArrivals;
  hipLaunchKernelGGL(balance_sequences_kernel, dim3(S, b.blocks), dim3(kSumThreads), 0, stream, part_p, part_c,
                     part_zn, T, E, k, seq, S, b.chunk, counts, tokens, losses, part, seq_z,
                     counted ? arrivals : nullptr);
  e = hipGetLastError();
  if (e != hipSuccess || counted) return e;
  hipLaunchKernelGGL(balance_losses_kernel, dim3(1), dim3(kSumThreads), 0, stream, part, seq_z, S, b.blocks, tokens,
                     losses);
  return hipGetLastError();
}

hipError_t launch_route_backward(const uint16_t* logits, const int32_t* ids, const float* gates, const float* dgates,
                                 int T, int E, int k, const int32_t* seq, int S, const int32_t* counts,
                                 const int32_t* tokens, const float* dlosses, void* dlogits, bool dlogits_f32,
                                 hipStream_t stream) {
  with_lanes(E, [&](auto lanes) {
    constexpr int L = decltype(lanes)::value;
    const int least = (T + (1 << 21) - 1) >> 21;  // a grid holds under 2^32 threads
    const int chunk = kRouteChunk<L> > least ? kRouteChunk<L> : least;
    const dim3 grid((T + chunk - 1) / chunk);
    auto with_out = [&](auto elem) {
      using O = decltype(elem);
      if (dlosses)
        hipLaunchKernelGGL((route_backward_kernel<L, O, true>), grid, dim3(kRouteThreads), 0, stream, logits, ids,
                           gates, dgates, T, E, k, seq, S, counts, tokens, dlosses, chunk,
                           static_cast<O*>(dlogits));
      else
        hipLaunchKernelGGL((route_backward_kernel<L, O, false>), grid, dim3(kRouteThreads), 0, stream, logits, ids,
                           gates, dgates, T, E, k, seq, S, counts, tokens, dlosses, chunk,
                           static_cast<O*>(dlogits));
    };
    if (dlogits_f32)
      with_out(float{});
    else
      with_out(uint16_t{});
  });
  return hipGetLastError();
}

}  // namespace mxfp4
