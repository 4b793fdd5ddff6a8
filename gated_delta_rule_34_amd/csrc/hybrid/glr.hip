// glr.hip -- the gated linear recurrence on gfx950: prompts, gradients, single tokens.
//
//   h_t = a_t h_{t-1} + b_t,  a_t = exp(-L_t),  b_t = w_t s(i_t) x_t,  w_t = sqrt(1 - a_t^2),
//   L_t = rate softplus(lambda) s(r_t)
// and backward, with c_t the gradient that reaches h_t from the tokens behind it and G_t = dy_t + c_t:
//   c_{t-1} = a_t G_t,  dx = w s(i) G,  di = x s(i) (1 - s(i)) w G,
//   L dL = G a L (u a / w - h_{t-1}) of u = s(i) x,  dr = L dL (1 - s(r)),
//   dlambda = sum L dL sigmoid(lambda) / softplus(lambda)
//
// Both directions are chains of affine maps h -> a h + b, which compose. A workgroup owns 128 bytes
// of channels (whole lines) and walks down its tokens in tiles of 128: each of 64 thread rows composes
// the maps of 2 tokens, four thread rows of a DPP row theirs by lane shifts, one wave (a channel per lane)
// the 16 such groups in LDS behind the carried state, and every thread then runs its tokens from the state in
// front of them. A map is kept as e = 1 - a and b (h -> h - e h + b, first e1 then e2: e1 + e2 - e1 e2): decays are close
// to one and e, unlike a, keeps its precision there (a state of 4096 tokens at decays around 0.99 is 2e-7 off, with a 7e-7);
// of a decay far below one a h is then formed to 2^-24 of h, not of itself.
//
// Every element is read and written once where one workgroup takes a whole sequence; where that
// leaves compute units idle, sequences are cut into segments, whose maps an extra pass over the inputs
// finds first.
#include "../gdn_common.h"
#include "../layer/rows.h"
#include "../layer/vec8.h"
#include "hybrid_internal.h"

namespace gdn {

constexpr int GNT = 512;           // threads
constexpr int GROWS = GNT / 8;     // thread rows: 8 threads hold the channels of a token
constexpr int GK = 2;              // tokens per thread and tile
constexpr int GTILE = GROWS * GK;  // tokens per tile
constexpr int GE = GNT / 32;       // groups of four thread rows

// V adjacent values of a row (16 bytes).
template <typename TI> constexpr int glr_v() { return 16 / (int)sizeof(TI); }
// A thread's piece of the rows of a tensor, from row `row` of a tile on (kNowhere: of no row).
template <typename TI> struct GlrView {
  const TI* p;
  int64_t rs;
  uint32_t rsb, voff;
  __device__ __forceinline__ GlrView(const void* base, int64_t stride, bool on, int row, int c)
      : p(static_cast<const TI*>(base)), rs(stride), rsb((uint32_t)stride * (uint32_t)sizeof(TI)) {
    voff = on ? (uint32_t)row * rsb + (uint32_t)c * (uint32_t)sizeof(TI) : kNowhere;
  }
  // The `rows` rows from t on (a tile's at the most).
  __device__ __forceinline__ __amdgpu_buffer_rsrc_t rows(int64_t t, int rows) const { return rows_rsrc(p + t * rs, (uint32_t)rows * rsb); }
  template <bool NT> __device__ __forceinline__ i32x4 load(__amdgpu_buffer_rsrc_t r, int k) const { return buf_ld16<NT>(r, voff + (uint32_t)k * rsb); }
  __device__ __forceinline__ void store(__amdgpu_buffer_rsrc_t r, int k, i32x4 v) const { buf_st16<true>(r, voff + (uint32_t)k * rsb, v); }
};
template <typename TI, int V> __device__ __forceinline__ void glr_cvt(i32x4 r, float (&v)[V]) {
  if constexpr (sizeof(TI) == 2) {
    const bf16x8 b = __builtin_bit_cast(bf16x8, r);
#pragma unroll
    for (int j = 0; j < V; ++j) v[j] = (float)b[j];
  } else {
    const f32x4 b = __builtin_bit_cast(f32x4, r);
#pragma unroll
    for (int j = 0; j < V; ++j) v[j] = b[j];
  }
}
template <typename TI, int V> __device__ __forceinline__ i32x4 glr_raw(const float (&v)[V]) {
  if constexpr (sizeof(TI) == 2) {
    bf16x8 b;
#pragma unroll
    for (int j = 0; j < V; ++j) b[j] = (__bf16)v[j];
    return __builtin_bit_cast(i32x4, b);
  } else {
    return __builtin_bit_cast(i32x4, f32x4{v[0], v[1], v[2], v[3]});
  }
}

// rate softplus(lambda), kept finite (an infinite exponent times a state would be NaN where a is zero).
__device__ __forceinline__ float glr_rate(float rate, float lam) {
  const float c = rate * softplusf(lam);
  return c > 0x1p100f ? 0x1p100f : c;
}

// exp(-L), for L >= 0.
template <typename TI> __device__ __forceinline__ float glr_exp(float L) {
  if constexpr (sizeof(TI) == 2) return __builtin_amdgcn_exp2f(L * -1.44269504f);
  else return expf(-L);
}
// 1 - exp(-L): its series up to L^6 below a quarter (the next term is 5e-8 of it). `deep` (wave-uniform): some L may
// be more; where no channel's rate is, the exponentials are left out.
template <typename TI, int V> __device__ __forceinline__ void one_minus_exp(const float (&L)[V], bool deep, float (&e)[V]) {
#pragma unroll
  for (int j = 0; j < V; ++j) {
    float p = fmaf(L[j], -1.f / 720.f, 1.f / 120.f);
    p = fmaf(L[j], p, -1.f / 24.f);
    p = fmaf(L[j], p, 1.f / 6.f);
    p = fmaf(L[j], p, -0.5f) * L[j];
    e[j] = fmaf(L[j], p, L[j]);
  }
  if (deep) {
    asm volatile("");  // (a branch, not eight exponentials for nothing)
#pragma unroll
    for (int j = 0; j < V; ++j) e[j] = L[j] < 0.25f ? e[j] : 1.f - glr_exp<TI>(L[j]);
  }
}

// w = sqrt(1 - a^2) of e = 1 - a. A w below 2^-63, whose square no float32 holds in full, may come out as less.
template <typename TI> __device__ __forceinline__ float glr_weight(float e) {
  if constexpr (sizeof(TI) == 2) return __builtin_amdgcn_sqrtf(e * (2.f - e));
  else return sqrtf(e * (2.f - e));
}
// 1 / w, which ends at 2^63 (L / w is then zero where L is).
template <typename TI> __device__ __forceinline__ float glr_inv_weight(float e) {
  const float w2 = fmaxf(e * (2.f - e), 0x1p-126f);
  if constexpr (sizeof(TI) == 2) return __builtin_amdgcn_rsqf(w2);
  else return 1.f / sqrtf(w2);
}

// (E, B) <- first (E1, B1), then (E, B).
__device__ __forceinline__ void glr_after(float E1, float B1, float& E, float& B) {
  B = fmaf(-E, B1, B1) + B;
  E = fmaf(-E1, E, E1) + E;
}

// x of the lane that CTRL names, zero where it lies outside the row of 16 (e = 0, b = 0: the map that changes nothing).
template <int CTRL> __device__ __forceinline__ float dpp_or0(float x) {
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), CTRL, 0xF, 0xF, true));
}
// The four thread rows of a DPP row: (E, B) composed with those in front of it (FWD, row_shr) or behind it
// (row_shl), and (Ex, Bx) that of the others alone.
template <bool FWD, int V> __device__ __forceinline__ void glr_scan4(float (&E)[V], float (&B)[V], float (&Ex)[V], float (&Bx)[V]) {
  constexpr int S4 = FWD ? 0x114 : 0x104, S8 = FWD ? 0x118 : 0x108;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    glr_after(dpp_or0<S4>(E[j]), dpp_or0<S4>(B[j]), E[j], B[j]);
    glr_after(dpp_or0<S8>(E[j]), dpp_or0<S8>(B[j]), E[j], B[j]);
    Ex[j] = dpp_or0<S4>(E[j]);
    Bx[j] = dpp_or0<S4>(B[j]);
  }
}

// A thread's place: lane bits 0, 1 and 4 name its piece of the channels, 2 and 3 its thread row among the four of its
// DPP row, bit 5 and the wave the group of four.
struct GlrLane {
  int cg, tt, g;
  bool first, last;  // of its four thread rows
  __device__ __forceinline__ GlrLane() {
    const int l = lane_id(), t4 = (l >> 2) & 3;
    cg = (l & 3) | ((l >> 4) & 1) << 2;
    g = wave_id() * 2 + (l >> 5);
    tt = g * 4 + t4;
    first = t4 == 0;
    last = t4 == 3;
  }
};

// Segment `slot` of the launch: tokens [t0, t1), the k-th of sequence n (rows [lo, hi)). Without a table: segment
// k of a packed sequence has slot lo / seg + n + k, below T_total / seg + N, and no two share one.
struct GlrSeg {
  int n, k;
  int64_t lo, hi, t0, t1;
};
__device__ __forceinline__ bool glr_seg(const GlrArgs& a, int slot, int seg, int per, GlrSeg& q) {
  if (!a.cu) {
    q.n = slot / per;
    q.k = slot - q.n * per;
    q.lo = (int64_t)q.n * a.T;
    q.hi = q.lo + a.T;
  } else {
    auto clamp = [&](int64_t v) { return v < 0 ? 0 : v > a.rows ? a.rows : v; };
    int l = 0;
    for (int n = a.N; n > 1;) {  // the largest n whose first slot is at most `slot`, 64 probes at a time
      const int stride = (n + 63) / 64, i = lane_id() * stride;
      const uint64_t m = __ballot(i < n && (int)((uint32_t)clamp(a.cu[l + (i < n ? i : 0)]) / (uint32_t)seg) + l + i <= slot);
      const int at = (m ? 63 - __builtin_clzll(m) : 0) * stride;
      l += at;
      n = n - at < stride ? n - at : stride;
    }
    q.n = __builtin_amdgcn_readfirstlane(l);
    q.lo = clamp(a.cu[q.n]);
    q.hi = clamp(a.cu[q.n + 1]);
    if (q.hi < q.lo) q.hi = q.lo;
    q.k = slot - (int)((uint32_t)q.lo / (uint32_t)seg) - q.n;
  }
  if (q.k < 0 || (q.k > 0 && (int64_t)q.k * seg >= q.hi - q.lo)) return false;
  q.t0 = q.lo + (int64_t)q.k * seg;
  q.t1 = q.t0 + seg < q.hi ? q.t0 + seg : q.hi;
  return true;
}

// Workgroup -> (segment slot, first channel): channel blocks run fastest, so that workgroups in flight read whole rows.
#define GLR_BEGIN                                                                        \
  constexpr int V = glr_v<TI>(), CB = 8 * V;                                             \
  const int cbn = (a.ch + CB - 1) / CB, slot = (int)blockIdx.x / cbn;                    \
  const int c0 = ((int)blockIdx.x - slot * cbn) * CB;                                    \
  const GlrLane me;                                                                      \
  const bool on = c0 + me.cg * V < a.ch;                                                 \
  const int c = on ? c0 + me.cg * V : 0, ci = c0 + lane_id();                            \
  const bool mine = lane_id() < CB && ci < a.ch; /* a channel of the scanning waves */   \
  float rate[V];                                                                         \
  bool deep = false;                                                                     \
  _Pragma("unroll") for (int j = 0; j < V; ++j) {                                        \
    rate[j] = glr_rate(a.rate, a.lam[c + j]);                                            \
    deep |= !(rate[j] < 0.25f);                                                          \
  }                                                                                      \
  deep = __any(deep)

// ------------------------------------------------------------------ maps of segments
// The map of each segment that another one continues from: forward every one but a sequence's last, backward
// every one but its first. A thread row takes a contiguous run of the tokens. [slot][E | B][ch].
template <typename TI, bool FWD> __global__ __launch_bounds__(GNT) void k_glr_map(GlrArgs a, int seg, int per) {
  __shared__ float sE[GE][8 * glr_v<TI>()], sB[GE][8 * glr_v<TI>()];
  GlrSeg q;
  GLR_BEGIN;
  if (!glr_seg(a, slot, seg, per, q) || (FWD ? q.t1 == q.hi : q.k == 0)) return;
  constexpr int U = 4;  // tokens of a run in flight; a run is a multiple of them
  const int run = (int)((q.t1 - q.t0 + GROWS * U - 1) / (GROWS * U)) * U;
  const bool fresh = FWD && a.fresh && q.k == 0 && a.fresh[q.n] != 0;
  float E[V], B[V];
#pragma unroll
  for (int j = 0; j < V; ++j) E[j] = B[j] = 0.f;
  // the segment's rows in steps of U: thread row tt takes row tt run + b (backward: run - U - b) of it
  const int64_t mine0 = q.t0 + (int64_t)me.tt * run;
  const TI *pr = static_cast<const TI*>(a.r) + c, *px = static_cast<const TI*>(FWD ? a.x : a.dy) + c, *pi = static_cast<const TI*>(a.i) + c;
  const int64_t x_rs = FWD ? a.x_rs : a.dy_rs;
  i32x4 rr[U], rx[U], ri[U];
  auto load = [&](int64_t t) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t row = t + u < q.t1 ? t + u : q.t1 - 1;
      rr[u] = *reinterpret_cast<const i32x4*>(pr + row * a.r_rs);
      rx[u] = *reinterpret_cast<const i32x4*>(px + row * x_rs);
      if constexpr (FWD) ri[u] = *reinterpret_cast<const i32x4*>(pi + row * a.i_rs);
    }
  };
  load(FWD ? mine0 : mine0 + run - U);
  for (int b = 0; b < run; b += U) {
    const int64_t t = FWD ? mine0 + b : mine0 + run - U - b;
    i32x4 cr[U], cx[U], ci4[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      cr[u] = rr[u];
      cx[u] = rx[u];
      if constexpr (FWD) ci4[u] = ri[u];
    }
    if (b + U < run) load(FWD ? t + U : t - U);
#pragma unroll
    for (int w = 0; w < U; ++w) {
      const int u = FWD ? w : U - 1 - w;
      if (t + u >= q.t1) continue;
      float r[V], x[V], iv[V], L[V], e[V];
      glr_cvt<TI, V>(cr[u], r);
      glr_cvt<TI, V>(cx[u], x);
      if constexpr (FWD) glr_cvt<TI, V>(ci4[u], iv);
#pragma unroll
      for (int j = 0; j < V; ++j) L[j] = rate[j] * sigmoidf<TI>(r[j]);
      one_minus_exp<TI, V>(L, deep, e);
      if (fresh && t + u == q.lo)
#pragma unroll
        for (int j = 0; j < V; ++j) e[j] = 1.f;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        if constexpr (FWD) B[j] = fmaf(1.f - e[j], B[j], glr_weight<TI>(e[j]) * (sigmoidf<TI>(iv[j]) * x[j]));
        else B[j] = (1.f - e[j]) * (B[j] + x[j]);
        E[j] = fmaf(-e[j], E[j], E[j]) + e[j];
      }
    }
  }
  float Ex[V], Bx[V];
  glr_scan4<FWD, V>(E, B, Ex, Bx);
  if (FWD ? me.last : me.first)
#pragma unroll
    for (int j = 0; j < V; ++j) {
      sE[me.g][me.cg * V + j] = E[j];
      sB[me.g][me.cg * V + j] = B[j];
    }
  __syncthreads();
  if (wave_id() == 0 && mine) {
    float e = 0.f, b = 0.f;
#pragma unroll
    for (int i = 0; i < GE; ++i) {
      const int g = FWD ? i : GE - 1 - i;
      float e2 = sE[g][lane_id()], b2 = sB[g][lane_id()];
      glr_after(e, b, e2, b2);
      e = e2;
      b = b2;
    }
    a.ws[(int64_t)slot * 2 * a.ch + ci] = e;
    a.ws[((int64_t)slot * 2 + 1) * a.ch + ci] = b;
  }
}

// ------------------------------------------------------------------ forward
template <typename TI, int K, bool SAVE> __global__ __launch_bounds__(GNT) void k_glr_fwd(GlrArgs a, int seg, int per) {
  __shared__ float sE[GE][8 * glr_v<TI>()], sB[GE][8 * glr_v<TI>()], sh[GE][8 * glr_v<TI>()];
  constexpr int TILE = GROWS * K, SUB = TILE / GTILE, GS = GE / SUB;  // states are saved every GTILE tokens
  GlrSeg q;
  GLR_BEGIN;
  if (!glr_seg(a, slot, seg, per, q)) return;
  const bool fresh = a.fresh && a.fresh[q.n] != 0;
  float h = 0.f;  // wave 0: the carried state of channel ci
  if (wave_id() == 0 && mine) {
    h = fresh || !a.h0 ? 0.f : a.h0[(int64_t)q.n * a.ch + ci];
    for (int s = slot - q.k; s < slot; ++s) {
      const float* m = a.ws + (int64_t)s * 2 * a.ch + ci;
      h = fmaf(-m[0], h, h) + m[a.ch];
    }
  }
  const GlrView<TI> vx(a.x, a.x_rs, on, me.tt * K, c), vr(a.r, a.r_rs, on, me.tt * K, c), vi(a.i, a.i_rs, on, me.tt * K, c),
      vy(a.y, a.y_rs, on, me.tt * K, c);
  auto left = [&](int64_t t) { return (int)(q.t1 - t < TILE ? q.t1 - t : TILE); };
  i32x4 rx[K], rr[K], ri[K];
  auto load = [&](int64_t t) {
    const int n = left(t);
    const auto sr = vr.rows(t, n), si = vi.rows(t, n), sx = vx.rows(t, n);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      rr[k] = vr.template load<true>(sr, k);
      ri[k] = vi.template load<true>(si, k);
      rx[k] = vx.template load<true>(sx, k);
    }
  };
  if (q.t0 < q.t1) load(q.t0);
  for (int64_t t = q.t0; t < q.t1; t += TILE) {
    float a1[K][V], b[K][V], E[V], B[V], Ex[V], Bx[V];  // a1 = 1 - e: what a map does to the tokens of this thread alone
    const bool plain = t + TILE <= q.t1 && !(fresh && t == q.lo);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float x[V], r[V], i[V], L[V], e[V];
      glr_cvt<TI, V>(rx[k], x);
      glr_cvt<TI, V>(rr[k], r);
      glr_cvt<TI, V>(ri[k], i);
#pragma unroll
      for (int j = 0; j < V; ++j) L[j] = rate[j] * sigmoidf<TI>(r[j]);
      one_minus_exp<TI, V>(L, deep, e);
      if (!plain) {
        const int64_t row = t + me.tt * K + k;
        if (fresh && row == q.lo)
#pragma unroll
          for (int j = 0; j < V; ++j) e[j] = 1.f;
        if (row >= q.t1)  // a token that changes nothing
#pragma unroll
          for (int j = 0; j < V; ++j) e[j] = x[j] = 0.f;
      }
#pragma unroll
      for (int j = 0; j < V; ++j) {
        b[k][j] = glr_weight<TI>(e[j]) * (sigmoidf<TI>(i[j]) * x[j]);
        a1[k][j] = 1.f - e[j];
        B[j] = k ? fmaf(a1[k][j], B[j], b[k][j]) : b[k][j];
        E[j] = k ? fmaf(-e[j], E[j], E[j]) + e[j] : e[j];
      }
    }
    if (t + TILE < q.t1) load(t + TILE);
    glr_scan4<true, V>(E, B, Ex, Bx);
    if (me.last)
#pragma unroll
      for (int j = 0; j < V; ++j) {
        sE[me.g][me.cg * V + j] = E[j];
        sB[me.g][me.cg * V + j] = B[j];
      }
    lds_barrier();
    if (wave_id() == 0 && lane_id() < CB) {
#pragma unroll
      for (int g = 0; g < GE; ++g) {
        if (SAVE && g % GS == 0 && mine && t + g / GS * GTILE < q.t1)
          a.sv[(q.lo / GTILE + q.n + (t - q.lo) / GTILE + g / GS) * a.ch + ci] = h;
        sh[g][lane_id()] = h;
        h = fmaf(-sE[g][lane_id()], h, h) + sB[g][lane_id()];
      }
    }
    lds_barrier();
    float y[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const float hc = sh[me.g][me.cg * V + j];
      y[j] = fmaf(-Ex[j], hc, hc) + Bx[j];
    }
    const auto out = vy.rows(t, left(t));
#pragma unroll
    for (int k = 0; k < K; ++k) {
#pragma unroll
      for (int j = 0; j < V; ++j) y[j] = fmaf(a1[k][j], y[j], b[k][j]);
      vy.store(out, k, glr_raw<TI, V>(y));
    }
  }
  if (a.hT && wave_id() == 0 && mine && q.t1 == q.hi) a.hT[(int64_t)q.n * a.ch + ci] = h;
}

// ------------------------------------------------------------------ backward
// Tiles from the last to the first; within a tile the states from its saved start and the gradients from
// those behind it side by side. Partials of dlambda: [slot][ch].
template <typename TI> __global__ __launch_bounds__(GNT) void k_glr_bwd(GlrArgs a, int seg, int per, float* part) {
  __shared__ float sE[GE][8 * glr_v<TI>()], sB[GE][8 * glr_v<TI>()], sC[GE][8 * glr_v<TI>()];
  __shared__ float sh[GE][8 * glr_v<TI>()], sg[GE][8 * glr_v<TI>()];
  GlrSeg q;
  GLR_BEGIN;
  if (!glr_seg(a, slot, seg, per, q)) {
    if (part && wave_id() == 0 && mine) part[(int64_t)slot * a.ch + ci] = 0.f;
    return;
  }
  const bool fresh = a.fresh && a.fresh[q.n] != 0;
  float cc = 0.f;  // wave 1: the gradient that flows into the tile's end
  if (wave_id() == 1 && mine) {
    cc = a.dhT ? a.dhT[(int64_t)q.n * a.ch + ci] : 0.f;
    const int segs = (int)((q.hi - q.lo + seg - 1) / seg);
    for (int s = slot - q.k + segs - 1; s > slot; --s) {
      const float* m = a.ws + (int64_t)s * 2 * a.ch + ci;
      cc = fmaf(-m[0], cc, cc) + m[a.ch];
    }
  }
  const GlrView<TI> vx(a.x, a.x_rs, on, me.tt * GK, c), vr(a.r, a.r_rs, on, me.tt * GK, c), vi(a.i, a.i_rs, on, me.tt * GK, c),
      vd(a.dy, a.dy_rs, on, me.tt * GK, c), ox(a.dx, a.dx_rs, on, me.tt * GK, c), orr(a.dr, a.dr_rs, on, me.tt * GK, c),
      oi(a.di, a.di_rs, on, me.tt * GK, c);
  auto left = [&](int64_t t) { return (int)(q.t1 - t < GTILE ? q.t1 - t : GTILE); };
  i32x4 rx[GK], rr[GK], ri[GK], rd[GK];
  auto load = [&](int64_t t) {
    const int n = left(t);
    const auto sr = vr.rows(t, n), si = vi.rows(t, n), sx = vx.rows(t, n), sd = vd.rows(t, n);
#pragma unroll
    for (int k = 0; k < GK; ++k) {
      rr[k] = vr.template load<true>(sr, k);
      ri[k] = vi.template load<true>(si, k);
      rx[k] = vx.template load<true>(sx, k);
      rd[k] = vd.template load<true>(sd, k);
    }
  };
  float dl[V];
#pragma unroll
  for (int j = 0; j < V; ++j) dl[j] = 0.f;
  const int64_t tiles = (q.t1 - q.t0 + GTILE - 1) / GTILE;
  if (tiles) load(q.t0 + (tiles - 1) * GTILE);
  for (int64_t tile = tiles - 1; tile >= 0; --tile) {
    const int64_t t = q.t0 + tile * GTILE;
    float hs = 0.f;  // wave 0: the tile's saved start
    if (wave_id() == 0 && mine) hs = a.sv[((q.lo / GTILE) + q.n + (t - q.lo) / GTILE) * a.ch + ci];
    const bool plain = t + GTILE <= q.t1 && !(fresh && t == q.lo);
    float e[GK][V], sr[GK][V], si[GK][V], E[V], B[V], Ex[V], Bx[V], F[V], C[V], Fx[V], Cx[V];
    i32x4 kx[GK], kd[GK];
#pragma unroll
    for (int k = 0; k < GK; ++k) {
      float x[V], r[V], i[V], L[V];
      glr_cvt<TI, V>(rx[k], x);
      glr_cvt<TI, V>(rr[k], r);
      glr_cvt<TI, V>(ri[k], i);
      kx[k] = rx[k];
      kd[k] = rd[k];
#pragma unroll
      for (int j = 0; j < V; ++j) {
        sr[k][j] = sigmoidf<TI>(r[j]);
        si[k][j] = sigmoidf<TI>(i[j]);
        L[j] = rate[j] * sr[k][j];
      }
      one_minus_exp<TI, V>(L, deep, e[k]);
      if (!plain) {
        const int64_t row = t + me.tt * GK + k;
        if (fresh && row == q.lo)
#pragma unroll
          for (int j = 0; j < V; ++j) e[k][j] = 1.f;
        if (row >= q.t1) {  // a token that changes nothing
          kx[k] = kd[k] = i32x4{0, 0, 0, 0};
#pragma unroll
          for (int j = 0; j < V; ++j) e[k][j] = x[j] = 0.f;
        }
      }
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float b = glr_weight<TI>(e[k][j]) * (si[k][j] * x[j]);
        B[j] = k ? fmaf(1.f - e[k][j], B[j], b) : b;
        E[j] = k ? fmaf(-e[k][j], E[j], E[j]) + e[k][j] : e[k][j];
      }
    }
#pragma unroll
    for (int k = GK - 1; k >= 0; --k) {
      float d[V];
      glr_cvt<TI, V>(kd[k], d);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        C[j] = (1.f - e[k][j]) * (k < GK - 1 ? C[j] + d[j] : d[j]);
        F[j] = E[j];
      }
    }
    if (tile > 0) load(t - GTILE);
    glr_scan4<true, V>(E, B, Ex, Bx);
    glr_scan4<false, V>(F, C, Fx, Cx);
    if (me.last)
#pragma unroll
      for (int j = 0; j < V; ++j) {
        sE[me.g][me.cg * V + j] = E[j];
        sB[me.g][me.cg * V + j] = B[j];
      }
    if (me.first)
#pragma unroll
      for (int j = 0; j < V; ++j) sC[me.g][me.cg * V + j] = C[j];
    lds_barrier();
    if (wave_id() == 0 && lane_id() < CB) {
#pragma unroll
      for (int g = 0; g < GE; ++g) {
        sh[g][lane_id()] = hs;
        hs = fmaf(-sE[g][lane_id()], hs, hs) + sB[g][lane_id()];
      }
    }
    if (wave_id() == 1 && lane_id() < CB) {
#pragma unroll
      for (int g = GE - 1; g >= 0; --g) {
        sg[g][lane_id()] = cc;
        cc = fmaf(-sE[g][lane_id()], cc, cc) + sC[g][lane_id()];
      }
    }
    lds_barrier();
    // What follows from these is formed anew: kept over the barriers it would take (and spill) more registers than there are.
#pragma unroll
    for (int k = 0; k < GK; ++k) {
      asm volatile("" : "+v"(kx[k]), "+v"(kd[k]));
#pragma unroll
      for (int j = 0; j < V; ++j) asm volatile("" : "+v"(e[k][j]), "+v"(sr[k][j]), "+v"(si[k][j]));
    }
    float hp[GK][V], cg[V];  // the state in front of each token, the gradient from behind
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const float hc = sh[me.g][me.cg * V + j], gc = sg[me.g][me.cg * V + j];
      hp[0][j] = fmaf(-Ex[j], hc, hc) + Bx[j];
      cg[j] = fmaf(-Fx[j], gc, gc) + Cx[j];
    }
#pragma unroll
    for (int k = 0; k + 1 < GK; ++k) {
      float x[V];
      glr_cvt<TI, V>(kx[k], x);
#pragma unroll
      for (int j = 0; j < V; ++j)
        hp[k + 1][j] = fmaf(1.f - e[k][j], hp[k][j], glr_weight<TI>(e[k][j]) * (si[k][j] * x[j]));
    }
    const auto tx = ox.rows(t, left(t)), tr = orr.rows(t, left(t)), ti = oi.rows(t, left(t));
#pragma unroll
    for (int k = GK - 1; k >= 0; --k) {
      const int64_t row = t + me.tt * GK + k;
      float x[V], d[V], dx[V], dr[V], di[V];
      glr_cvt<TI, V>(kx[k], x);
      glr_cvt<TI, V>(kd[k], d);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float G = cg[j] + d[j], u = si[k][j] * x[j], L = rate[j] * sr[k][j], a1 = 1.f - e[k][j];
        float al = a1;  // a to its own last bits
        if (deep && !(fresh && row == q.lo)) al = L < 0.25f ? a1 : glr_exp<TI>(L);
        const float rw = glr_inv_weight<TI>(e[k][j]), du = e[k][j] * (2.f - e[k][j]) * rw * G;
        dx[j] = si[k][j] * du;
        di[j] = u * (1.f - si[k][j]) * du;
        // L dL; a and L first, whose product stays finite
        const float LdL = (al * L) * G * fmaf(u * al, rw, -hp[k][j]);
        dr[j] = LdL * (1.f - sr[k][j]);
        dl[j] += row < q.t1 ? LdL : 0.f;
        cg[j] = a1 * G;
      }
      ox.store(tx, k, glr_raw<TI, V>(dx));
      orr.store(tr, k, glr_raw<TI, V>(dr));
      oi.store(ti, k, glr_raw<TI, V>(di));
    }
  }
  if (a.dh0 && wave_id() == 1 && mine && q.k == 0) a.dh0[(int64_t)q.n * a.ch + ci] = fresh ? 0.f : cc;
  if (part) {
    __syncthreads();
#pragma unroll
    for (int j = 0; j < V; ++j) {  // the four thread rows, then the groups
      dl[j] += dpp_or0<0x114>(dl[j]);
      dl[j] += dpp_or0<0x118>(dl[j]);
      if (me.last) sE[me.g][me.cg * V + j] = dl[j];
    }
    __syncthreads();
    if (wave_id() == 0 && mine) {
      float s = 0.f;
#pragma unroll
      for (int g = 0; g < GE; ++g) s += sE[g][lane_id()];
      const float lam = a.lam[ci], sp = softplusf(lam);
      // sigmoid / softplus; both vanish together, and with them the sum
      part[(int64_t)slot * a.ch + ci] = sp > 0.f ? s * ((1.f / (1.f + expf(-lam))) / sp) : 0.f;
    }
  }
}

// ------------------------------------------------------------------ one token
template <typename TI> __global__ __launch_bounds__(64) void k_glr_decode(GlrArgs a) {
  const int c = (int)(blockIdx.y * 64 + threadIdx.x) * 8, n = (int)blockIdx.x;
  if (c >= a.ch) return;
  const int slot = a.idx ? a.idx[n] : n;
  if (slot < 0 || slot >= a.n_slots) return;
  const bool fresh = a.fresh && a.fresh[n] != 0;
  float* st = a.state + (int64_t)slot * a.ch + c;
  const Raw8<TI> rx = ldraw8<false, TI>((const TI*)a.x + (int64_t)n * a.x_rs + c);
  const Raw8<TI> rr = ldraw8<false, TI>((const TI*)a.r + (int64_t)n * a.r_rs + c);
  const Raw8<TI> ri = ldraw8<false, TI>((const TI*)a.i + (int64_t)n * a.i_rs + c);
  const F8 lam = ld8<float>(a.lam + c);
  F8 h = fresh ? zero8() : ld8<float>(st);
  const F8 x = cvt8<TI>(rx), r = cvt8<TI>(rr), i = cvt8<TI>(ri);
  float L[8], e[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) L[j] = glr_rate(a.rate, lam.v[j]) * sigmoidf<TI>(r.v[j]);
  one_minus_exp<TI, 8>(L, true, e);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float u = sigmoidf<TI>(i.v[j]) * x.v[j];
    h.v[j] = fresh ? u : fmaf(-e[j], h.v[j], h.v[j]) + glr_weight<TI>(e[j]) * u;
  }
  st8<float>(st, h);
  st8<TI>((TI*)a.y + (int64_t)n * a.y_rs + c, h);
}

// ------------------------------------------------------------------ launches
struct GlrPlan {
  int seg, per, slots, cbn;
  bool cut;  // some sequence may have more than one segment
};
static GlrPlan glr_plan(const GlrArgs& a, int dtype) {
  GlrPlan p;
  const int CB = dtype == 0 ? 32 : 64;
  p.cbn = (a.ch + CB - 1) / CB;
  const int64_t longest = a.cu ? a.rows : a.T;
  int64_t seg = (longest + GTILE - 1) / GTILE * GTILE;
  if ((int64_t)p.cbn * a.N < 256 || a.cu) {
    const int64_t want = ((int64_t)p.cbn * a.rows / 512 + GTILE - 1) / GTILE * GTILE;
    const int64_t s = want < 512 ? 512 : want;
    if (s < seg) seg = s;
  }
  if (seg < GTILE) seg = GTILE;
  p.seg = (int)seg;
  p.per = a.cu ? 0 : (int)((a.T + seg - 1) / seg);
  if (!a.cu && p.per < 1) p.per = 1;
  p.slots = a.cu ? (int)(a.rows / seg) + a.N : a.N * p.per;
  p.cut = longest > seg;
  return p;
}

size_t glr_fwd_ws_bytes(const GlrArgs& a, int dtype) {
  const GlrPlan p = glr_plan(a, dtype);
  return p.cut ? (size_t)p.slots * 2 * a.ch * sizeof(float) : 0;
}
size_t glr_bwd_ws_bytes(const GlrArgs& a, int dtype) {
  const GlrPlan p = glr_plan(a, dtype);
  return (size_t)p.slots * a.ch * sizeof(float) * (p.cut ? 3 : 1);
}
// A tile has the slot of a segment of one tile.
size_t glr_saved_bytes(const GlrArgs& a) { return ((size_t)(a.rows / GTILE) + a.N) * a.ch * sizeof(float); }

template <typename TI> static hipError_t glr_forward(const GlrArgs& a, int dtype, hipStream_t s) {
  const GlrPlan p = glr_plan(a, dtype);
  const unsigned grid = (unsigned)p.slots * (unsigned)p.cbn;
  if (grid == 0) return hipSuccess;
  if (p.cut) {
    traced("k_glr_map", s, [&] { k_glr_map<TI, true><<<grid, GNT, 0, s>>>(a, p.seg, p.per); });
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  traced("k_glr_fwd", s, [&] {
    if (a.sv) k_glr_fwd<TI, 4, true><<<grid, GNT, 0, s>>>(a, p.seg, p.per);
    else k_glr_fwd<TI, 4, false><<<grid, GNT, 0, s>>>(a, p.seg, p.per);
  });
  return hipGetLastError();
}

template <typename TI> static hipError_t glr_backward(const GlrArgs& a, int dtype, hipStream_t s) {
  const GlrPlan p = glr_plan(a, dtype);
  const unsigned grid = (unsigned)p.slots * (unsigned)p.cbn;
  hipError_t e = hipSuccess;
  if (p.cut && grid) {
    traced("k_glr_map", s, [&] { k_glr_map<TI, false><<<grid, GNT, 0, s>>>(a, p.seg, p.per); });
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  float* part = a.dlam ? a.ws + (p.cut ? (int64_t)p.slots * 2 * a.ch : 0) : nullptr;
  if (grid) traced("k_glr_bwd", s, [&] { k_glr_bwd<TI><<<grid, GNT, 0, s>>>(a, p.seg, p.per, part); });
  e = hipGetLastError();
  if (e == hipSuccess && part) e = launch_colsum(part, p.slots, a.ch, ColsumOut{{a.dlam, nullptr, nullptr}}, 1, s);
  return e;
}

hipError_t launch_glr_forward(const GlrArgs& a, int dtype, hipStream_t s) {
  return dtype == 0 ? glr_forward<float>(a, dtype, s) : glr_forward<__bf16>(a, dtype, s);
}
hipError_t launch_glr_backward(const GlrArgs& a, int dtype, hipStream_t s) {
  return dtype == 0 ? glr_backward<float>(a, dtype, s) : glr_backward<__bf16>(a, dtype, s);
}
hipError_t launch_glr_decode(const GlrArgs& a, int dtype, hipStream_t s) {
  if (a.N == 0) return hipSuccess;
  const dim3 grid((unsigned)a.N, (unsigned)((a.ch / 8 + 63) / 64));
  traced("k_glr_decode", s, [&] {
    if (dtype == 0) k_glr_decode<float><<<grid, 64, 0, s>>>(a);
    else k_glr_decode<__bf16><<<grid, 64, 0, s>>>(a);
  });
  return hipGetLastError();
}

}  // namespace gdn
