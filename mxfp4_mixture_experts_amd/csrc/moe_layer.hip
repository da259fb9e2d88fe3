// A whole expert layer for a few tokens in two launches, for gfx950:
//
//   xn = bf16(x r w_norm), logits = xn . router^T + bias (fp32), the k largest and their
//   softmax; act = bf16(swiglu(gate_up[e] . xn + bias)) for every chosen expert;
//   y = (x +) sum over slots of gate (down[e] . act + bias).
//
// The layer has two points where every workgroup needs what all others made (the
// routing; the activations).  The second is the border of the launches.  At the
// first each workgroup of the first launch makes the routing itself: it reads the
// router's E rows from L2 (at E = 32, H = 2880 184 KB, about 2.6 us with all 256 CUs
// at it), which costs less than a launch and its latency, and no workgroup ever
// waits for another.
//
// Both launches stream the chosen experts' weights once for all tokens: a unit is 4
// weight rows of an expert, 16 lanes a row, lane j of a row blocks j, j + 16, ... (256
// contiguous bytes of a row a load).  The units of all chosen experts are spread
// evenly over 256 workgroups of 12 waves, and a wave has the next unit's loads
// under way while it multiplies.  A block becomes 32 exact bf16 weights and meets
// each of its expert's tokens in bf16 dot products with fp32 sums; the tokens' rows
// lie in LDS by pieces of 8 elements ([piece of a block][block]), so that 16
// lanes' reads are contiguous.

#include "kernels.h"
#include "common.h"
#include "fp4_dot.h"

namespace mxfp4 {
namespace {

constexpr int kWaves = 12, kThreads = kWaves * 64;
constexpr int kGroups = 256;  // workgroups: one a CU
constexpr int kIns = 6;       // blocks a lane takes at a time: 96 blocks of a row
constexpr int kSpan = 16 * kIns;
constexpr int kPieces = 6;    // 8-element pieces of a router row a lane holds
constexpr int kRouted = 3;    // router rows a wave holds
constexpr int kMaxRows = kLayerMaxT * kLayerMaxTopK;

__device__ __forceinline__ float row16_sum(float v) {  // over the 16 lanes of a row, fixed order
  v += __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), 0xB1, 0xF, 0xF, true));   // l ^ 1
  v += __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), 0x4E, 0xF, 0xF, true));   // l ^ 2
  v += __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), 0x141, 0xF, 0xF, true));  // within 8
  v += __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), 0x140, 0xF, 0xF, true));  // within 16
  return v;
}
__device__ __forceinline__ float lane_value(float v, int l) {
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), l));
}
__device__ __forceinline__ float wave_total(float v) {
  v = row16_sum(v);
  return (lane_value(v, 0) + lane_value(v, 16)) + (lane_value(v, 32) + lane_value(v, 48));
}
__device__ __forceinline__ float wave_max(float v) {
  v = fmaxf(v, __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), 0xB1, 0xF, 0xF, true)));
  v = fmaxf(v, __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), 0x4E, 0xF, 0xF, true)));
  v = fmaxf(v, __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), 0x141, 0xF, 0xF, true)));
  v = fmaxf(v, __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), 0x140, 0xF, 0xF, true)));
  return fmaxf(fmaxf(lane_value(v, 0), lane_value(v, 16)), fmaxf(lane_value(v, 32), lane_value(v, 48)));
}

// One lane's blocks of a unit: the four weight rows are 16 lanes each.
struct Unit {
  uint4 w[kIns];
  uint32_t s[kIns];
};
__device__ __forceinline__ void load_unit(Unit& u, const uint8_t* blocks, const uint8_t* scales, size_t row, int KB,
                                          int b0, int j) {
  const uint4* w = reinterpret_cast<const uint4*>(blocks) + row * KB;
  const uint8_t* s = scales + row * KB;
#pragma unroll
  for (int i = 0; i < kIns; i++) {
    const int b = min(b0 + 16 * i + j, KB - 1);  // past the row: its last block, masked when multiplied
    u.w[i] = load_nt(w + b);
    u.s[i] = s[b];
  }
}
// sum over this lane's blocks of weights times the staged row (4 pieces of KB blocks)
__device__ __forceinline__ float unit_dot(const Unit& u, const uint4* row, int KB, int b0, int j, float a) {
#pragma unroll
  for (int i = 0; i < kIns; i++) {
    const int b = b0 + 16 * i + j;
    if (b0 + 16 * i < KB) {
      const int c = min(b, KB - 1);
      a = block_dot(u.w[i], b < KB ? ~0u : 0u, e8m0_value(u.s[i]), row[c], row[KB + c], row[2 * KB + c],
                    row[3 * KB + c], a);
    }
  }
  return a;
}

// The experts with tokens, from slot_of[t][e] (the slot, -1 if none): their list, and
// each one's tokens as bits.  One wave.
__device__ __forceinline__ void list_experts(const int8_t* slot_of, int T, int E, int lane, int* list, uint32_t* tokens,
                                             int* count) {
  uint32_t mask = 0;
  for (int t = 0; t < T; t++)
    if (lane < E && slot_of[t * 64 + lane] >= 0) mask |= 1u << t;
  const uint64_t used = wave_ballot(mask != 0);
  if (mask) {
    const int at = lanes_below(used);
    list[at] = lane;
    tokens[at] = mask;
  }
  if (lane == 0) *count = __popcll(used);
}

template <bool F32>
__device__ __forceinline__ void load8(const void* x, size_t i, float (&v)[8]) {
  if (F32) {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(x) + i);
    const float4 a = p[0], b = p[1];
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  } else {
    const uint4 d = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(x) + i);
    const uint32_t w[4] = {d.x, d.y, d.z, d.w};
#pragma unroll
    for (int j = 0; j < 4; j++) {
      v[2 * j] = __uint_as_float(w[j] << 16);
      v[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
    }
  }
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) { return f32_to_bf16_any(lo) | f32_to_bf16_any(hi) << 16; }

// Norm, router, routing, and the gate/up projection through the activation.
template <bool F32>
__global__ __launch_bounds__(kThreads) void layer_gate_up_kernel(MoeLayerArgs a) {
  extern __shared__ __attribute__((aligned(16))) uint4 xs[];  // [T][4][H / 32]
  __shared__ float logits[kLayerMaxT * 64];
  __shared__ int8_t slot_of[kLayerMaxT * 64];
  __shared__ int list[64];
  __shared__ uint32_t tokens[64];
  __shared__ int count;
  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int KB = a.H >> 5;
  const int H8 = a.H >> 3;

  // this wave's first router rows are under way during the norm
  uint4 wr[kRouted][kPieces];
  auto load_router = [&](int e0, int p0) {
#pragma unroll
    for (int r = 0; r < kRouted; r++) {
      const uint4* w = reinterpret_cast<const uint4*>(a.router_w) + (size_t)min(e0 + r * kWaves, a.E - 1) * H8;
#pragma unroll
      for (int i = 0; i < kPieces; i++) wr[r][i] = w[min(p0 + 64 * i + lane, H8 - 1)];
    }
  };
  load_router(wave, 0);

  // norm: a wave a token; piece p of 8 elements is piece p % 4 of block p / 4
  for (int t = wave; t < a.T; t += kWaves) {
    float r = 1.f;
    if (a.w_norm) {
      float ss = 0.f;
      for (int p = lane; p < H8; p += 64) {
        float v[8];
        load8<F32>(a.x, (size_t)t * a.H + 8 * p, v);
#pragma unroll
        for (int j = 0; j < 8; j++) ss = fmaf(v[j], v[j], ss);
      }
      r = 1.0f / sqrtf(wave_total(ss) / (float)a.H + a.eps);
    }
    for (int p = lane; p < H8; p += 64) {
      uint4 o;
      if (a.w_norm) {
        float v[8], w[8];
        load8<F32>(a.x, (size_t)t * a.H + 8 * p, v);
        load8<false>(a.w_norm, 8 * p, w);
#pragma unroll
        for (int j = 0; j < 8; j++) v[j] = v[j] * r * w[j];
        o = make_uint4(pack2(v[0], v[1]), pack2(v[2], v[3]), pack2(v[4], v[5]), pack2(v[6], v[7]));
      } else {
        o = reinterpret_cast<const uint4*>(a.x)[(size_t)t * H8 + p];
      }
      xs[(size_t)t * 4 * KB + (p & 3) * KB + (p >> 2)] = o;
    }
  }
  for (int i = tid; i < a.T * 64; i += kThreads) slot_of[i] = -1;
  __syncthreads();

  // router: wave w takes experts w, w + kWaves, ..., kRouted at a time
  const bool whole = H8 <= 64 * kPieces;  // a row is held whole
  for (int e0 = wave; e0 < a.E; e0 += kRouted * kWaves) {
    if (whole && e0 != wave) load_router(e0, 0);
    for (int t = 0; t < a.T; t++) {
      float acc[kRouted] = {};
      for (int p0 = 0; p0 < H8; p0 += 64 * kPieces) {
        if (!whole) load_router(e0, p0);
#pragma unroll
        for (int i = 0; i < kPieces; i++) {
          const int p = p0 + 64 * i + lane;
          if (p < H8) {
            const uint4 xv = xs[(size_t)t * 4 * KB + (p & 3) * KB + (p >> 2)];
#pragma unroll
            for (int r = 0; r < kRouted; r++) acc[r] = dot8(wr[r][i], xv, acc[r]);
          }
        }
      }
#pragma unroll
      for (int r = 0; r < kRouted; r++) {
        const int e = e0 + r * kWaves;
        const float l = wave_total(acc[r]);
        if (lane == 0 && e < a.E) logits[t * 64 + e] = l + (a.router_b ? bf16_bits_to_f32(a.router_b[e]) : 0.f);
      }
    }
  }
  __syncthreads();

  // routing: a wave a token, lane e expert e; k rounds of the largest logit, the lowest index among equals
  for (int t = wave; t < a.T; t += kWaves) {
    const float l = lane < a.E ? logits[t * 64 + lane] : -INFINITY;
    const bool bad = wave_ballot(!(l < INFINITY)) != 0;  // a NaN or an infinity has no softmax
    bool open = lane < a.E;
    float top = 0.f, mine = 0.f;  // lane s: exp(logit of slot s - the largest)
    int id = -1;                  // lane s: the expert of slot s
    float sum = 0.f;
    for (int s = 0; s < a.k && !bad; s++) {
      const float m = wave_max(open ? l : -INFINITY);
      const int e = __builtin_ctzll(wave_ballot(open && l == m));
      if (s == 0) top = m;
      const float g = m == top ? 1.f : expf(m - top);
      sum += g;
      if (lane == e) {
        open = false;
        slot_of[t * 64 + e] = (int8_t)s;
      }
      if (lane == s) {
        id = e;
        mine = g;
      }
    }
    if (blockIdx.x == 0 && lane < a.k) {
      const float g = bad ? 0.f : mine / sum;
      a.ws_ids[t * a.k + lane] = id;
      a.ws_gates[t * a.k + lane] = g;
      if (a.ids) a.ids[t * a.k + lane] = id;
      if (a.gates) a.gates[t * a.k + lane] = g;
    }
  }
  __syncthreads();
  if (wave == 0) list_experts(slot_of, a.T, a.E, lane, list, tokens, &count);
  __syncthreads();

  // units of 4 rows (two gate and up pairs) of the chosen experts
  const int per = a.F >> 1;
  const int units = count * per;
  const int u1 = (int)((long long)units * (blockIdx.x + 1) / gridDim.x);
  int u = (int)((long long)units * blockIdx.x / gridDim.x) + wave;
  const int q = lane >> 4, j = lane & 15;
  auto row_of = [&](int v) {
    const int i = v / per;
    return (size_t)list[i] * (2 * a.F) + 4 * (v - i * per) + q;
  };
  Unit cur, next;
  if (u < u1) load_unit(cur, a.gu, a.gu_scales, row_of(u), KB, 0, j);
  for (; u < u1; u += kWaves) {
    if (u + kWaves < u1) load_unit(next, a.gu, a.gu_scales, row_of(u + kWaves), KB, 0, j);
    const int i = u / per;
    const int e = list[i], r0 = 4 * (u - i * per);
    const float bias = a.gu_bias ? bf16_bits_to_f32(a.gu_bias[(size_t)e * 2 * a.F + r0 + q]) : 0.f;
    for (uint32_t m = __builtin_amdgcn_readfirstlane(tokens[i]); m; m &= m - 1) {
      const int t = __builtin_ctz(m);
      const uint4* row = xs + (size_t)t * 4 * KB;
      float p = unit_dot(cur, row, KB, 0, j, 0.f);
      for (int b0 = kSpan; b0 < KB; b0 += kSpan) {
        Unit more;
        load_unit(more, a.gu, a.gu_scales, (size_t)e * 2 * a.F + r0 + q, KB, b0, j);
        p = unit_dot(more, row, KB, b0, j, p);
      }
      p = row16_sum(p) + bias;
      const float up = __shfl_xor(p, 16, 64);
      if (j == 0 && (q & 1) == 0) {
        const int s = slot_of[t * 64 + e];
        a.act[(size_t)(t * a.k + s) * a.F + (r0 >> 1) + (q >> 1)] = (uint16_t)f32_to_bf16_any(swiglu(p, up));
      }
    }
    cur = next;
  }
}

// The down projection, the combine in slot order and the residual.
template <bool F32>
__global__ __launch_bounds__(kThreads) void layer_down_kernel(MoeLayerArgs a, int lds_rows, int max_quads) {
  // staged rows [lds_rows][4][F / 32], then the outputs [max_quads][4][T k]
  extern __shared__ __attribute__((aligned(16))) uint4 as[];
  __shared__ int8_t slot_of[kLayerMaxT * 64];
  __shared__ int list[64];
  __shared__ uint32_t tokens[64];
  __shared__ int count;
  __shared__ float gates[kMaxRows];
  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int KB = a.F >> 5, F8 = a.F >> 3;
  const int R = a.T * a.k;
  float* const outs = reinterpret_cast<float*>(as + (size_t)lds_rows * F8);
  for (int i = tid; i < a.T * 64; i += kThreads) slot_of[i] = -1;
  __syncthreads();
  for (int r = tid; r < R; r += kThreads) {
    const int t = r / a.k;
    const int e = a.ws_ids[r];
    gates[r] = a.ws_gates[r];
    if ((unsigned)e < (unsigned)a.E) slot_of[t * 64 + e] = (int8_t)(r - t * a.k);
  }
  __syncthreads();
  if (wave == 0) list_experts(slot_of, a.T, a.E, lane, list, tokens, &count);
  __syncthreads();

  const int quads = a.H >> 2;
  const int q0 = (int)((long long)quads * blockIdx.x / gridDim.x);
  const int nq = (int)((long long)quads * (blockIdx.x + 1) / gridDim.x) - q0;
  const int q = lane >> 4, j = lane & 15;
  // as many experts at a time as their tokens' rows fit
  for (int first = 0; first < count;) {
    int end = first, rows = 0;
    while (end < count) {
      const int n = __popc(__builtin_amdgcn_readfirstlane(tokens[end]));
      if (rows + n > lds_rows) break;
      rows += n;
      end++;
    }
    const int units = (end - first) * nq;
    auto row_of = [&](int v) {
      const int i = v / nq;
      return (size_t)list[first + i] * a.H + 4 * (q0 + v - i * nq) + q;
    };
    Unit cur, next;
    int u = wave;
    if (u < units) load_unit(cur, a.down, a.down_scales, row_of(u), KB, 0, j);
    // the rows, expert by expert, token by token
    {
      int at = 0;
      for (int i = first; i < end; i++) {
        const int e = list[i];
        for (uint32_t m = __builtin_amdgcn_readfirstlane(tokens[i]); m; m &= m - 1, at++) {
          const int t = __builtin_ctz(m);
          const uint4* src = reinterpret_cast<const uint4*>(a.act + (size_t)(t * a.k + slot_of[t * 64 + e]) * a.F);
          for (int p = tid; p < F8; p += kThreads) as[(size_t)at * F8 + (p & 3) * KB + (p >> 2)] = src[p];
        }
      }
    }
    __syncthreads();
    for (; u < units; u += kWaves) {
      if (u + kWaves < units) load_unit(next, a.down, a.down_scales, row_of(u + kWaves), KB, 0, j);
      const int i = u / nq, quad = u - i * nq;
      const int e = list[first + i];
      int at = 0;
      for (int b = first; b < first + i; b++) at += __popc(tokens[b]);
      const float bias = a.down_bias ? bf16_bits_to_f32(a.down_bias[(size_t)e * a.H + 4 * (q0 + quad) + q]) : 0.f;
      for (uint32_t m = __builtin_amdgcn_readfirstlane(tokens[first + i]); m; m &= m - 1, at++) {
        const int t = __builtin_ctz(m);
        const uint4* row = as + (size_t)at * F8;
        float p = unit_dot(cur, row, KB, 0, j, 0.f);
        for (int b0 = kSpan; b0 < KB; b0 += kSpan) {
          Unit more;
          load_unit(more, a.down, a.down_scales, row_of(u), KB, b0, j);
          p = unit_dot(more, row, KB, b0, j, p);
        }
        p = row16_sum(p) + bias;
        if (j == 0) outs[(quad * 4 + q) * R + t * a.k + slot_of[t * 64 + e]] = p;
      }
      cur = next;
    }
    __syncthreads();
    first = end;
  }
  for (int i = tid; i < nq * 4 * a.T; i += kThreads) {
    const int t = i / (nq * 4), c = i - t * nq * 4;
    const size_t at = (size_t)t * a.H + 4 * q0 + c;
    float h = 0.f;
    for (int s = 0; s < a.k; s++) {
      const float g = gates[t * a.k + s];
      if (g != 0.f) h = fmaf(g, outs[c * R + t * a.k + s], h);  // (a slot without an expert has gate 0)
    }
    if (a.residual) h += F32 ? static_cast<const float*>(a.x)[at] : bf16_bits_to_f32(static_cast<const uint16_t*>(a.x)[at]);
    if (a.y_f32) static_cast<float*>(a.y)[at] = h;
    else static_cast<uint16_t*>(a.y)[at] = (uint16_t)f32_to_bf16_any(h);
  }
}

size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }

}  // namespace

size_t moe_layer_workspace_bytes(int T, int k, int F) {
  const size_t R = (size_t)T * k;
  return 2 * align256(R * 4) + align256(R * F * 2);
}

hipError_t launch_moe_layer(MoeLayerArgs a, bool x_f32, void* workspace, hipStream_t stream) {
  const size_t R = (size_t)a.T * a.k;
  uint8_t* const ws = static_cast<uint8_t*>(workspace);
  a.ws_ids = reinterpret_cast<int32_t*>(ws);
  a.ws_gates = reinterpret_cast<float*>(ws + align256(R * 4));
  a.act = reinterpret_cast<uint16_t*>(ws + 2 * align256(R * 4));
  const int quads = a.H / 4;
  const int groups = quads < kGroups ? quads : kGroups;
  const int max_quads = (quads + groups - 1) / groups;
  const size_t outs = (size_t)max_quads * 4 * R * 4;
  // every row that one expert can have, more where they fit
  const size_t fit = (kLayerLds - outs) / ((size_t)a.F * 2);
  const int lds_rows = (int)(fit < R ? fit : R);
  static DynLdsLimit limits[4] = {{reinterpret_cast<const void*>(layer_gate_up_kernel<false>), kLayerLds},
                                  {reinterpret_cast<const void*>(layer_gate_up_kernel<true>), kLayerLds},
                                  {reinterpret_cast<const void*>(layer_down_kernel<false>), kLayerLds},
                                  {reinterpret_cast<const void*>(layer_down_kernel<true>), kLayerLds}};
  hipError_t e = limits[x_f32].ensure();
  if (e == hipSuccess) e = limits[2 + x_f32].ensure();
  if (e != hipSuccess) return e;
  const size_t up_lds = (size_t)a.T * a.H * 2, down_lds = (size_t)lds_rows * a.F * 2 + outs;
  auto up = x_f32 ? layer_gate_up_kernel<true> : layer_gate_up_kernel<false>;
  auto down = x_f32 ? layer_down_kernel<true> : layer_down_kernel<false>;
  hipLaunchKernelGGL(up, dim3(kGroups), dim3(kThreads), up_lds, stream, a);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(down, dim3(groups), dim3(kThreads), down_lds, stream, a, lds_rows, max_quads);
  return hipGetLastError();
}

}  // namespace mxfp4
