// A whole expert layer for a few tokens in three launches, for gfx950:
//
//   router  xn = bf16(x r w_norm), logits = xn . router^T + bias (fp32): a workgroup an
//           expert, a wave a token, which norms the token itself;
//   gate/up the k largest logits and their softmax (by every workgroup for itself), then
//           act = bf16(swiglu(gate_up[e] . xn + bias)) for every chosen expert;
//   down    y = (x +) sum over slots of gate (down[e] . act + bias).
//
// The borders of the launches are the two points where every workgroup needs what all
// others made; no workgroup waits for another.  Moving the norm and the router out of the
// gate/up launch (where each workgroup did its own) took one token of H = F = 2880, E = 32,
// k = 4 from 27.3 to 25.1 us: 256 CUs read the same 184 KB at 17 bytes a clock each.  Now
// 24 to 27 us from HBM, as the experts fall, and 74 to 79 for eight tokens.
//
// Both projections stream the chosen experts' weights once for all tokens, by items of 16
// weight rows x 4 blocks (lane: row lane % 16, block lane / 16), a wave's items in
// registers ahead of their use.  A block becomes 32 exact bf16 weights
// (v_cvt_scalef32_pk_bf16_fp4) and one MFMA for each quarter of the blocks multiplies
// them by up to 16 tokens' rows: the work of an item does not grow with the tokens.
// K is split over the waves alike whatever the tokens are, and a token's sums hold
// nothing of the others: its outputs are the same bits alone and in any batch.

#include "kernels.h"
#include "common.h"

namespace mxfp4 {
namespace {

typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));

constexpr int kWaves = 12, kThreads = kWaves * 64;
constexpr int kGroups = 256;       // workgroups of gate/up: one a CU
constexpr int kRouterWaves = 8;    // router: tokens at a time
constexpr int kPieces = 6;         // router: 16-byte pieces of a row that a lane holds
constexpr uint32_t kPast = 0x80000000u;  // an offset past every buffer: the load returns zeros

// 2^(s - 127): s = 0 is the subnormal 2^-127
__device__ __forceinline__ float e8m0_value(uint32_t s) { return __uint_as_float(max(s << 23, 0x00400000u)); }

template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), CTRL, 0xF, 0xF, true));
}
__device__ __forceinline__ float lane_value(float v, int l) {
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), l));
}
__device__ __forceinline__ float row16_total(float v) {  // of the 16 lanes of a row, in a fixed order
  v += dpp<0xB1>(v);    // l ^ 1
  v += dpp<0x4E>(v);    // l ^ 2
  v += dpp<0x141>(v);   // within 8
  v += dpp<0x140>(v);   // within 16
  return v;
}
__device__ __forceinline__ float wave_total(float v) {
  v = row16_total(v);
  return (lane_value(v, 0) + lane_value(v, 16)) + (lane_value(v, 32) + lane_value(v, 48));
}
__device__ __forceinline__ float wave_max(float v) {
  v = fmaxf(v, dpp<0xB1>(v));
  v = fmaxf(v, dpp<0x4E>(v));
  v = fmaxf(v, dpp<0x141>(v));
  v = fmaxf(v, dpp<0x140>(v));
  return fmaxf(fmaxf(lane_value(v, 0), lane_value(v, 16)), fmaxf(lane_value(v, 32), lane_value(v, 48)));
}

// 16 weight rows x 4 blocks times the 16 tokens' inputs of those blocks, added to acc
__device__ __forceinline__ f32x4_t item_mma(const u32x4_t w, uint32_t scale, const uint4* x, f32x4_t acc) {
  const float sf = e8m0_value(scale);
#pragma unroll
  for (int d = 0; d < 4; d++) {
    const bf16x2_t a0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[d], sf, 0);
    const bf16x2_t a1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[d], sf, 1);
    const bf16x2_t a2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[d], sf, 2);
    const bf16x2_t a3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[d], sf, 3);
    const bf16x8_t a = {a0[0], a0[1], a1[0], a1[1], a2[0], a2[1], a3[0], a3[1]};
    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, __builtin_bit_cast(bf16x8_t, x[d]), acc, 0, 0, 0);
  }
  return acc;
}

// Where a lane finds its blocks b, b + 4, ... of a row: in a unit's codes and scales, zeros
// past the row, and among the row's inputs, past it the pieces from x_past on (finite
// numbers wherever the row's are: they meet the zeros).
template <int C>
struct Places {
  uint32_t w[C], s[C];
  int x[C];
  __device__ __forceinline__ void set(int row, int b, int KB, int x_past) {
#pragma unroll
    for (int j = 0; j < C; j++) {
      const bool in = b + 4 * j < KB;
      s[j] = in ? row * KB + b + 4 * j : kPast;
      w[j] = in ? (row * KB + b + 4 * j) * 16 : kPast;
      x[j] = in ? (b + 4 * j) * 4 : x_past;
    }
  }
};

// A wave's part of a unit's K: C items held in registers; each is loaded again, for the next
// unit, as soon as it is used.
template <int C>
struct Stream {
  u32x4_t w[C];
  uint32_t s[C];
  __amdgpu_buffer_rsrc_t wsrc, ssrc;  // the unit's 16 rows; of no bytes if there is none: zeros
  __device__ __forceinline__ void open(const uint8_t* blocks, const uint8_t* scales, size_t first_row, int KB,
                                       bool any) {
    wsrc = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(blocks + first_row * KB * 16), (short)0,
                                             any ? 16 * KB * 16 : 0, 0x00020000);
    ssrc = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(scales + first_row * KB), (short)0,
                                             any ? 16 * KB : 0, 0x00020000);
  }
  // Items j and j + 1: the two halves of 128 bytes of a row, one after the other.  They stay in
  // the order of their use: the codes moved before all scales, the first item waited for all.
  __device__ __forceinline__ void load2(int j, const Places<C>& at) {
    w[j] = __builtin_amdgcn_raw_buffer_load_b128(wsrc, at.w[j], 0, 0);
    w[j + 1] = __builtin_amdgcn_raw_buffer_load_b128(wsrc, at.w[j + 1], 0, 0);
    s[j] = __builtin_amdgcn_raw_buffer_load_b8(ssrc, at.s[j], 0, 0);
    s[j + 1] = __builtin_amdgcn_raw_buffer_load_b8(ssrc, at.s[j + 1], 0, 0);
    __builtin_amdgcn_sched_barrier(0);
  }
  __device__ __forceinline__ f32x4_t use(const Places<C>& at, const uint4* x) {
    f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < C; j += 2) {
      acc = item_mma(w[j], s[j], x + at.x[j], acc);
      acc = item_mma(w[j + 1], s[j + 1], x + at.x[j + 1], acc);
      load2(j, at);
    }
    return acc;
  }
};

// sum of v over this lane and those below
__device__ __forceinline__ int wave_prefix(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, true);   // row shifted right by 1, 2, 4, 8
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);  // lane 15 to row 1, lane 47 to row 3
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);  // lane 31 to rows 2 and 3
  return v;
}

// The experts with tokens, the i-th in lane i (past the last: the others, without tokens).  The
// activations' rows stand expert by expert, token by token.
struct Experts {
  int expert;
  uint32_t tokens;  // as bits
  int rows_to;      // rows of the experts up to this one
};
__device__ __forceinline__ Experts list_experts(uint32_t mask, int lane) {
  const uint64_t used = wave_ballot(mask != 0);
  const int at = mask ? lanes_below(used) : __popcll(used) + lanes_below(~used);
  Experts x;
  x.expert = __builtin_amdgcn_ds_permute(at * 4, lane);
  x.tokens = (uint32_t)__builtin_amdgcn_ds_permute(at * 4, (int)mask);
  x.rows_to = wave_prefix(__popc(x.tokens));
  return x;
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  return __builtin_bit_cast(uint32_t, bf16x2_t{(__bf16)lo, (__bf16)hi});
}
__device__ __forceinline__ void unpack8(const uint4 d, float (&v)[8]) {
  const uint32_t w[4] = {d.x, d.y, d.z, d.w};
#pragma unroll
  for (int j = 0; j < 4; j++) {
    v[2 * j] = __uint_as_float(w[j] << 16);
    v[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
  }
}

// 16-byte pieces from one row in LDS to the next: 4 for a block, and one by which four rows'
// reads of 4 blocks each meet 16 different banks of 16 bytes
__host__ __device__ constexpr int row_stride(int KB) { return 4 * KB + 1; }

// Rows of bf16 into LDS, 16-byte piece p of row r at r RS + p: a wave takes 64 pieces of a
// row at a time, four such under way.  64 pieces behind the last row take what is not there.
struct Rows {
  __amdgpu_buffer_rsrc_t src;
  int pieces, spans, RS, spare, wave, lane;  // of a row; 64s of them; a row in LDS; the pieces behind
  u32x4_t v[4];
  int to[4];
  __device__ __forceinline__ void open(const void* rows, int bytes, int n8, int lds_rows, int w, int l) {
    src = __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(rows), (short)0, bytes, 0x00020000);
    pieces = n8;
    spans = (n8 + 63) >> 6;
    RS = row_stride(n8 >> 2);
    spare = lds_rows * RS + l;
    wave = w;
    lane = l;
  }
  // parts u0, u0 + kWaves, ... of the rows from row0 on
  __device__ __forceinline__ void load(int u0, int parts, int row0) {
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const int u = u0 + i * kWaves, r = u / spans, p = (u - r * spans) * 64 + lane;
      const bool there = u < parts && p < pieces;
      uint32_t from = there ? (uint32_t)((row0 + r) * pieces + p) * 16 : kPast;
      to[i] = there ? r * RS + p : spare;
      asm("" : "+v"(from), "+v"(to[i]));  // both chosen here: no branch around the load
      v[i] = __builtin_amdgcn_raw_buffer_load_b128(src, from, 0, 0);
    }
  }
  __device__ __forceinline__ void store(uint4* lds) {
#pragma unroll
    for (int i = 0; i < 4; i++) lds[to[i]] = __builtin_bit_cast(uint4, v[i]);
  }
  __device__ __forceinline__ void all(uint4* lds, int parts, int row0) {
    for (int u0 = wave; u0 < parts; u0 += 4 * kWaves) {
      load(u0, parts, row0);
      store(lds);
    }
  }
};

// Norm and router.  ONCE: a lane holds its pieces of a row, else it goes over the row again.
template <bool F32, bool NORM, bool ONCE>
__global__ __launch_bounds__(kRouterWaves * 64) void layer_router_kernel(MoeLayerArgs a) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int H8 = a.H >> 3, e = blockIdx.x;
  const uint4* const router = reinterpret_cast<const uint4*>(a.router_w) + (size_t)e * H8;
  const uint16_t* const bias = a.router_b ? a.router_b + e : a.router_w;  // (read and not used without one)
  for (int t = wave; t < a.T; t += kRouterWaves) {
    const uint4* const x = reinterpret_cast<const uint4*>(a.x) + (size_t)t * H8 * (F32 ? 2 : 1);
    uint4 raw[kPieces][F32 ? 2 : 1], wn[kPieces], rw[kPieces];
    auto load_x = [&](int p0) {
#pragma unroll
      for (int i = 0; i < kPieces; i++) {
        const int p = min(p0 + 64 * i + lane, H8 - 1);
        raw[i][0] = x[p * (F32 ? 2 : 1)];
        if (F32) raw[i][F32 ? 1 : 0] = x[p * 2 + 1];
      }
    };
    auto load_w = [&](int p0) {
#pragma unroll
      for (int i = 0; i < kPieces; i++) {
        const int p = min(p0 + 64 * i + lane, H8 - 1);
        if (NORM) wn[i] = reinterpret_cast<const uint4*>(a.w_norm)[p];
        rw[i] = router[p];
      }
    };
    auto values = [&](int i, float (&v)[8]) {
      if (F32) {
        const uint4 lo = raw[i][0], hi = raw[i][F32 ? 1 : 0];
        const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
        for (int j = 0; j < 8; j++) v[j] = __uint_as_float(w[j]);
      } else {
        unpack8(raw[i][0], v);
      }
    };
    const bool keeps = NORM && t % a.E == e;  // one workgroup writes a token's row
    float ss = 0.f, r = 1.f, acc = 0.f;
    auto square = [&](int p0) {
#pragma unroll
      for (int i = 0; i < kPieces; i++) {
        float v[8], s = 0.f;
        values(i, v);
#pragma unroll
        for (int j = 0; j < 8; j++) s = fmaf(v[j], v[j], s);
        ss += p0 + 64 * i + lane < H8 ? s : 0.f;
      }
    };
    auto dot = [&](int p0) {
#pragma unroll
      for (int i = 0; i < kPieces; i++) {
        const int p = p0 + 64 * i + lane;
        uint4 o = raw[i][0];
        if (NORM) {
          float v[8], w[8];
          values(i, v);
          unpack8(wn[i], w);
#pragma unroll
          for (int j = 0; j < 8; j++) v[j] = v[j] * r * w[j];
          o = make_uint4(pack2(v[0], v[1]), pack2(v[2], v[3]), pack2(v[4], v[5]), pack2(v[6], v[7]));
        }
        const uint32_t xv[4] = {o.x, o.y, o.z, o.w}, wv[4] = {rw[i].x, rw[i].y, rw[i].z, rw[i].w};
        float s = 0.f;
#pragma unroll
        for (int j = 0; j < 4; j++)
          s = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2_t, xv[j]), __builtin_bit_cast(bf16x2_t, wv[j]),
                                              s, false);
        acc += p < H8 ? s : 0.f;
        if (keeps && p < H8) reinterpret_cast<uint4*>(a.ws_xn)[(size_t)t * H8 + p] = o;
      }
    };
    load_x(0);
    const uint32_t bias_bits = *bias;
    if (ONCE) {
      load_w(0);
      __builtin_amdgcn_sched_barrier(0);  // every load is on its way before the first is waited for
      if (NORM) square(0);
    } else if (NORM) {
      square(0);
      for (int p0 = 64 * kPieces; p0 < H8; p0 += 64 * kPieces) {
        load_x(p0);
        square(p0);
      }
    }
    if (NORM) r = rsqrtf(fmaf(wave_total(ss), a.inv_H, a.eps));  // (as moe_norm: right for a subnormal eps too)
    if (ONCE) {
      dot(0);
    } else {
      for (int p0 = 0; p0 < H8; p0 += 64 * kPieces) {
        load_x(p0);
        load_w(p0);
        dot(p0);
      }
    }
    acc = wave_total(acc);
    if (lane == 0) a.ws_logits[t * 64 + e] = a.router_b ? acc + bf16_bits_to_f32(bias_bits) : acc;
  }
}

// Routing, and the gate/up projection through the activation.
template <int C, int TEAMS>
__global__ __launch_bounds__(kThreads) void layer_gate_up_kernel(MoeLayerArgs a) {
  // the tokens' rows, 64 pieces, then two rounds of the teams' partial sums
  extern __shared__ __attribute__((aligned(16))) uint4 xs[];
  __shared__ uint32_t tokens[64];
  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int col = lane & 15, q = lane >> 4;
  const int KB = a.H >> 5, RS = row_stride(KB);
  float4* const part = reinterpret_cast<float4*>(xs + a.T * RS + 64);
  const int xrow = min(col, a.T - 1) * RS;  // (columns past the tokens repeat the last)

  const float first_logit = lane < a.E && wave < a.T ? a.ws_logits[wave * 64 + lane] : 0.f;
  if (tid < 64) tokens[tid] = 0;
  if (tid < 4) xs[a.T * RS + tid] = make_uint4(0, 0, 0, 0);  // what stands past a row's end (x may be infinite)
  Rows rows;
  rows.open(a.w_norm ? a.ws_xn : a.x, a.T * a.H * 2, a.H >> 3, a.T, wave, lane);
  rows.load(wave, a.T * rows.spans, 0);
  __syncthreads();

  // routing: a wave a token, lane e expert e; k rounds of the largest logit, the lowest index among equals
  for (int t = wave; t < a.T; t += kWaves) {
    const float given = t == wave ? first_logit : a.ws_logits[t * 64 + min(lane, a.E - 1)];
    const float l = lane < a.E ? given : -INFINITY;
    const bool bad = wave_ballot(!(l < INFINITY)) != 0;  // a NaN or an infinity has no softmax
    bool open = lane < a.E, mine = false;
    float top = 0.f, of_slot = 0.f;  // the largest logit; lane s: that of slot s
    int id = -1;                     // lane s: the expert of slot s
    for (int s = 0; s < a.k && !bad; s++) {
      const float m = wave_max(open ? l : -INFINITY);
      const int e = __builtin_ctzll(wave_ballot(open && l == m));
      if (s == 0) top = m;
      if (lane == e) {
        open = false;
        mine = true;
      }
      if (lane == s) {
        id = e;
        of_slot = m;
      }
    }
    if (mine) atomicOr(&tokens[lane], 1u << t);
    if (blockIdx.x == 0) {
      // (of two equal infinities the difference is no number, the quotient 1)
      const float g = id < 0 ? 0.f : of_slot == top ? 1.f : expf(of_slot - top);
      const float all = wave_total(g);
      const float ge = !mine ? 0.f : l == top ? 1.f : expf(l - top);
      a.ws_gates[t * 64 + lane] = bad ? 0.f : ge / all;
      if (lane < a.k) {
        a.ws_ids[t * a.k + lane] = id;
        if (a.ids) a.ids[t * a.k + lane] = id;
        if (a.gates) a.gates[t * a.k + lane] = bad ? 0.f : g / all;
      }
    }
  }
  rows.store(xs);
  for (int u0 = wave + 4 * kWaves; u0 < a.T * rows.spans; u0 += 4 * kWaves) {
    rows.load(u0, a.T * rows.spans, 0);
    rows.store(xs);
  }
  __syncthreads();
  const Experts x = list_experts(tokens[lane], lane);
  const int count = __popcll(wave_ballot(x.tokens != 0));
  if (blockIdx.x == 0 && wave == 0) {
    a.ws_experts[lane] = x.expert;
    a.ws_experts[64 + lane] = (int)x.tokens;
    a.ws_experts[128 + lane] = x.rows_to;
  }

  // Units of 16 rows (8 gate and up pairs) of the chosen experts, spread evenly over the
  // workgroups; a workgroup's go to its teams in turn, one a round.
  const int per = a.F >> 3, units = count * per;  // (per >= 4)
  const int u0 = (unsigned)units * blockIdx.x / gridDim.x;  // (units <= 2^16, 256 workgroups)
  const int mine = (int)((unsigned)units * (blockIdx.x + 1) / gridDim.x) - u0;
  if (mine == 0) return;
  constexpr int kTeam = kWaves / TEAMS;
  const int team = wave / kTeam, part_of = wave - team * kTeam;
  const int rounds = (mine + TEAMS - 1) / TEAMS;
  Stream<C> st;
  Places<C> at;
  at.set(col, part_of * 4 * C + q, KB, a.T * RS - xrow);
  int ld_i = (u0 + team) / per, ld_tile = u0 + team - ld_i * per, ld_left = mine - team;
  auto next_unit = [&]() {
    const size_t unit = (size_t)__builtin_amdgcn_readlane(x.expert, min(ld_i, 63)) * per + ld_tile;
    st.open(a.gu, a.gu_scales, unit * 16, KB, ld_left > 0);
    ld_left -= TEAMS;
    ld_tile += TEAMS;
    if (ld_tile >= per) {
      ld_tile -= per;
      ld_i++;
    }
  };
  next_unit();
#pragma unroll
  for (int j = 0; j < C; j += 2) st.load2(j, at);
  // the sum over a team, the bias and the activation: a thread has a unit's pair of rows and a token
  const int out_pair = tid & 7, out_t = (tid >> 3) & 15, out_team = min(tid >> 7, TEAMS - 1);
  const int out_tr = min(out_t, a.T - 1);
  int out_i = (u0 + out_team) / per, out_tile = u0 + out_team - out_i * per;
  const uint16_t* const bias = a.gu_bias ? a.gu_bias : a.router_w;  // (read and not used without one)
  for (int r = 0; r < rounds; r++) {
    const bool out = tid < TEAMS * 128 && out_t < a.T && r * TEAMS + out_team < mine;
    // its bias is loaded ahead of the next round's weights: loads return in order
    const int oi = min(out_i, count - 1), e = __shfl(x.expert, oi, 64), row = out_tile * 16 + 2 * out_pair;
    const uint32_t its = __shfl(x.tokens, oi, 64);
    const int rows_to = __shfl(x.rows_to, oi, 64);
    const size_t bias_at = a.gu_bias ? (size_t)e * 2 * a.F + row : 0;
    const uint32_t gate_bias = bias[bias_at], up_bias = bias[bias_at + 1];
    next_unit();
    const f32x4_t acc = st.use(at, xs + xrow);
    float4* const mine_of = part + (r & 1) * kWaves * a.T * 4;
    if (col < a.T) mine_of[(wave * a.T + col) * 4 + q] = make_float4(acc[0], acc[1], acc[2], acc[3]);
    __syncthreads();
    if (out && (its >> out_tr & 1)) {
      float gate = a.gu_bias ? bf16_bits_to_f32(gate_bias) : 0.f, up = a.gu_bias ? bf16_bits_to_f32(up_bias) : 0.f;
      float2 d[kTeam];
#pragma unroll
      for (int p = 0; p < kTeam; p++)
        d[p] = reinterpret_cast<const float2*>(mine_of)[((out_team * kTeam + p) * a.T + out_tr) * 8 + out_pair];
#pragma unroll
      for (int p = 0; p < kTeam; p++) {
        gate += d[p].x;
        up += d[p].y;
      }
      const int pos = rows_to - __popc(its >> out_tr);
      a.act[(size_t)pos * a.F + (row >> 1)] = (uint16_t)f32_to_bf16_any(swiglu(gate, up));
    }
    out_tile += TEAMS;
    if (out_tile >= per) {
      out_tile -= per;
      out_i++;
    }
  }
}

// The down projection, the combine and the residual: a workgroup owns 16 output columns of
// all tokens.  A team of its waves shares K; with more teams than one (a short K) team i takes
// the experts whose number is i mod TEAMS, whatever the others are.  One expert's weights are
// under way a team; the activations lie in LDS, as many experts' at a time as fit (one's at
// least: T rows).
template <int C, int TEAMS>
__global__ __launch_bounds__(kThreads) void layer_down_kernel(MoeLayerArgs a, int lds_rows) {
  extern __shared__ __attribute__((aligned(16))) uint4 as[];  // as the tokens' rows above
  __shared__ float gates[kLayerMaxT * 64];
  __shared__ float4 part[kWaves * kLayerMaxT * 4];
  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int col = lane & 15, q = lane >> 4;
  const int KB = a.F >> 5, F8 = a.F >> 3, RS = row_stride(KB);
  Experts x;
  x.expert = a.ws_experts[lane];
  x.tokens = (uint32_t)a.ws_experts[64 + lane];
  x.rows_to = a.ws_experts[128 + lane];
  // what is added at the end is loaded ahead: thread (token, column); the first four slots' biases
  const int out_t = min(tid >> 4, a.T - 1), out_c = blockIdx.x * 16 + (tid & 15);
  const size_t out_at = (size_t)out_t * a.H + out_c;
  int id[4];
#pragma unroll
  for (int s = 0; s < 4; s++) id[s] = a.ws_ids[out_t * a.k + min(s, a.k - 1)];
  float gate_in[2];  // T * 64 <= 1024 of them
#pragma unroll
  for (int i = 0; i < 2; i++) gate_in[i] = a.ws_gates[min(tid + i * kThreads, a.T * 64 - 1)];

  const int count = __popcll(wave_ballot(x.tokens != 0));
  // the activations' rows of the experts that fit
  Rows rows;
  rows.open(a.act, a.T * a.k * a.F * 2, F8, lds_rows, wave, lane);
  int first = 0, last = 0, row0 = 0, parts = 0;
  auto next_rows = [&]() {
    first = last;
    row0 = first ? __builtin_amdgcn_readlane(x.rows_to, first - 1) : 0;
    last = min(count, __popcll(wave_ballot(x.rows_to - row0 <= lds_rows)));  // at least one more
    parts = (__builtin_amdgcn_readlane(x.rows_to, max(last, 1) - 1) - row0) * rows.spans;
  };
  next_rows();

  constexpr int kTeam = kWaves / TEAMS;
  const int team = wave / kTeam;
  Stream<C> st;
  Places<C> at;
  at.set(col, (wave - team * kTeam) * 4 * C + q, KB, (KB - 1) * 4);  // (an activation is finite, or NaN)
  uint64_t left = wave_ballot(x.tokens != 0 && x.expert % TEAMS == team);  // the team's, as bits of the list
  auto open = [&]() {
    const int e = __builtin_amdgcn_readlane(x.expert, left ? __builtin_ctzll(left) : 0);
    st.open(a.down, a.down_scales, (size_t)e * a.H + (size_t)blockIdx.x * 16, KB, left != 0);
  };
  const uint16_t* const bias = a.down_bias ? a.down_bias : a.router_w;  // (read and not used without one)
  auto bias_of = [&](int e) { return (uint32_t)bias[a.down_bias ? (size_t)max(e, 0) * a.H + out_c : 0]; };
  uint32_t bias_bits[4], x_bits;
  auto load_weights = [&]() {
    open();
#pragma unroll
    for (int j = 0; j < C; j += 2) st.load2(j, at);
#pragma unroll
    for (int s = 0; s < 4; s++) bias_bits[s] = bias_of(id[s]);
    // (the 32 bits that hold x: x is 16-byte aligned and H even)
    x_bits = static_cast<const uint32_t*>(a.x)[a.x_f32 ? out_at : out_at >> 1];
  };
  // A wave that cannot issue its weights' loads for the others' waits: a few rows come before
  // them; more would keep memory waiting for their latency, and go behind.
  if (parts <= 4 * kWaves) {
    rows.load(wave, parts, 0);
    rows.store(as);
    load_weights();
  } else {
    load_weights();
    rows.all(as, parts, 0);
  }
#pragma unroll
  for (int i = 0; i < 2; i++)
    if (tid + i * kThreads < a.T * 64) gates[tid + i * kThreads] = gate_in[i];
  f32x4_t y = {0.f, 0.f, 0.f, 0.f};
  const int tcol = min(col, a.T - 1);
  __syncthreads();
  for (;;) {
    while (left && __builtin_ctzll(left) < last) {
      const int i = __builtin_ctzll(left);
      left &= left - 1;
      const uint32_t m = __builtin_amdgcn_readlane(x.tokens, i);
      const bool has = (m >> col) & 1;
      // this token's row; where it does not have the expert, some row, not used
      const int row = has ? __builtin_amdgcn_readlane(x.rows_to, i) - row0 - __popc(m >> col) : 0;
      open();
      const f32x4_t acc = st.use(at, as + row * RS);
      const float gt = gates[tcol * 64 + __builtin_amdgcn_readlane(x.expert, i)], g = has ? gt : 0.f;
#pragma unroll
      for (int r = 0; r < 4; r++) y[r] = g != 0.f ? fmaf(g, acc[r], y[r]) : y[r];  // (0 adds nothing)
    }
    if (last >= count) break;
    next_rows();
    __syncthreads();
    rows.all(as, parts, row0);
    __syncthreads();
  }
  if (col < a.T) part[(wave * a.T + col) * 4 + q] = make_float4(y[0], y[1], y[2], y[3]);
  __syncthreads();
  if (tid < a.T * 16) {
    float sum = 0.f, d[kWaves];
#pragma unroll
    for (int p = 0; p < kWaves; p++) d[p] = reinterpret_cast<const float*>(part)[(p * a.T + out_t) * 16 + (tid & 15)];
#pragma unroll
    for (int p = 0; p < kWaves; p++) sum += d[p];
    auto add_bias = [&](int e, uint32_t b) {
      const float g = e >= 0 && a.down_bias ? gates[out_t * 64 + e] : 0.f;
      if (g != 0.f) sum = fmaf(g, bf16_bits_to_f32(b), sum);
    };
#pragma unroll
    for (int s = 0; s < 4; s++)
      if (s < a.k) add_bias(id[s], bias_bits[s]);
    for (int s = 4; s < a.k; s++) {
      const int e = a.ws_ids[out_t * a.k + s];
      add_bias(e, bias_of(e));
    }
    const float xv = __uint_as_float(a.x_f32 ? x_bits : out_at & 1 ? x_bits & 0xffff0000u : x_bits << 16);
    const float h = a.residual ? xv + sum : sum;
    if (a.y_f32) static_cast<float*>(a.y)[out_at] = h;
    else static_cast<uint16_t*>(a.y)[out_at] = (uint16_t)f32_to_bf16_any(h);
  }
}

// items that a wave of a team holds for its share of KB blocks, by twos
int items_of(int KB, int team) { return ((KB + 4 * team - 1) / (4 * team) + 1) / 2 * 2; }

template <bool F32, bool NORM>
hipError_t launch_router(const MoeLayerArgs& a, hipStream_t stream) {
  const dim3 grid(a.E), block((a.T < kRouterWaves ? a.T : kRouterWaves) * 64);
  if (a.H / 8 <= 64 * kPieces) hipLaunchKernelGGL((layer_router_kernel<F32, NORM, true>), grid, block, 0, stream, a);
  else hipLaunchKernelGGL((layer_router_kernel<F32, NORM, false>), grid, block, 0, stream, a);
  return hipGetLastError();
}

template <int C, int TEAMS>
hipError_t launch_up(const MoeLayerArgs& a, hipStream_t stream) {
  static DynLdsLimit limit(reinterpret_cast<const void*>(layer_gate_up_kernel<C, TEAMS>), kLayerUpLds);
  const size_t lds = ((size_t)a.T * row_stride(a.H / 32) + 64) * 16 + (size_t)2 * kWaves * 64 * a.T;
  if (lds > (size_t)kLayerUpLds) return hipErrorInvalidConfiguration;
  const hipError_t e = limit.ensure();
  if (e != hipSuccess) return e;
  const int R = a.T * a.k, most = (R < a.E ? R : a.E) * (a.F / 8);  // units of all experts that the tokens can reach
  hipLaunchKernelGGL((layer_gate_up_kernel<C, TEAMS>), dim3(most < kGroups ? most : kGroups), dim3(kThreads), lds,
                     stream, a);
  return hipGetLastError();
}
hipError_t launch_up(const MoeLayerArgs& a, hipStream_t stream) {
  // Three teams of 4 waves while a wave's share of K is 6 items at most, else one of 12 (the layer,
  // one token / eight: H = 288, F = 2880 16.0 / 40 us, with one team 18.7 / 52; H = F = 1440 14.7 / 33 to
  // 15.5 / 39; 2048 20.7 / 55 to 20.4 / 68; 2880 23.5 / 75 to 23.1 / 70; beyond, with one team, 4096 44 / 148,
  // with three of 8 items 42 / 147; 3584 x 2880 28 / 86 to 26 / 80)
  const int KB = a.H / 32, C = items_of(KB, kWaves / 3);
  return C == 2                      ? launch_up<2, 3>(a, stream)
         : C == 4                    ? launch_up<4, 3>(a, stream)
         : C == 6                    ? launch_up<6, 3>(a, stream)
         : items_of(KB, kWaves) <= 4 ? launch_up<4, 1>(a, stream)
                                     : launch_up<6, 1>(a, stream);
}

template <int C, int TEAMS>
hipError_t launch_down(const MoeLayerArgs& a, hipStream_t stream) {
  static DynLdsLimit limit(reinterpret_cast<const void*>(layer_down_kernel<C, TEAMS>), kLayerDownLds);
  const size_t row = (size_t)row_stride(a.F / 32) * 16;
  const int fit = (int)(((size_t)kLayerDownLds - 64 * 16) / row), R = a.T * a.k;
  if (fit < a.T) return hipErrorInvalidConfiguration;
  const hipError_t e = limit.ensure();
  if (e != hipSuccess) return e;
  const int rows = fit < R ? fit : R;
  hipLaunchKernelGGL((layer_down_kernel<C, TEAMS>), dim3(a.H / 16), dim3(kThreads),
                     rows * row + 64 * 16, stream, a, rows);
  return hipGetLastError();
}

size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }

}  // namespace

size_t moe_layer_workspace_bytes(int T, int H, int k, int F) {
  return T ? 1024 + (size_t)T * (2 * 64 * 4 + kLayerMaxTopK * 4) + align256((size_t)T * H * 2) +
                 align256((size_t)T * k * F * 2)
           : 0;
}

hipError_t launch_moe_layer(MoeLayerArgs a, void* workspace, hipStream_t stream) {
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  auto take = [&](size_t bytes) {
    uint8_t* const p = ws;
    ws += bytes;
    return p;
  };
  a.ws_experts = reinterpret_cast<int32_t*>(take(1024));
  a.ws_logits = reinterpret_cast<float*>(take((size_t)a.T * 64 * 4));
  a.ws_gates = reinterpret_cast<float*>(take((size_t)a.T * 64 * 4));
  a.ws_ids = reinterpret_cast<int32_t*>(take((size_t)a.T * kLayerMaxTopK * 4));
  a.ws_xn = reinterpret_cast<uint16_t*>(take(align256((size_t)a.T * a.H * 2)));
  a.act = reinterpret_cast<uint16_t*>(ws);
  hipError_t e = !a.w_norm ? launch_router<false, false>(a, stream)
                 : a.x_f32 ? launch_router<true, true>(a, stream)
                           : launch_router<false, true>(a, stream);
  if (e == hipSuccess) e = launch_up(a, stream);
  if (e != hipSuccess) return e;
  // Three teams of 4 waves, or two of 6, while their waves hold K in two items, else one of 12
  // (with one alone 16 tokens of F = 1024, E = 64, k = 8 took 72.8 us for 63.3, 8 of F = 1440, E = 32,
  // k = 4 35.8 for 32.7; with more at F = 2880 eight tokens took 75 to 76 us for 73.3: the teams'
  // experts are seldom as many).
  const int KB = a.F / 32, C = items_of(KB, kWaves);  // (6 at most)
  return items_of(KB, kWaves / 3) == 2   ? launch_down<2, 3>(a, stream)
         : items_of(KB, kWaves / 2) == 2 ? launch_down<2, 2>(a, stream)
         : C == 2                        ? launch_down<2, 1>(a, stream)
         : C == 4                        ? launch_down<4, 1>(a, stream)
                                         : launch_down<6, 1>(a, stream);
}

}  // namespace mxfp4
