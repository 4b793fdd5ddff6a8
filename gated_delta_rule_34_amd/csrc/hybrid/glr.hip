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
// front of them. A map is kept as e = 1 - a and b (h -> h - e h + b, first e1 then e2: e2 + e1 (1 - e2)): decays are close
// to one and e, unlike a, keeps its precision there; of a decay far below one a h is then formed to 2^-24 of h, not of itself.
//
// Every element is read and written once where one workgroup takes a whole sequence; where that
// leaves compute units idle, sequences are cut into segments, whose maps an extra pass over the inputs
// finds first. Measured (bf16): 4 x 4096 tokens x 2560 forward 95 us, backward 176 us, bound by the gates (five
// instructions of a quarter of the rate and some 30 others a value, in the 160 compute units that have a workgroup); one prompt of
// 16384 x 4096 77 us for the maps and 91 for the states, bound by HBM (5.2 and 5.9 TB/s); float32, 1336
// ragged tokens x 1032, 8 us for the maps, 16 forward and 22 backward: the latency of a few tiles one after the other.
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

// V adjacent values of a row (16 bytes), and the same as float32.
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
  __device__ __forceinline__ i32x4 load(__amdgpu_buffer_rsrc_t r, int k) const { return buf_ld16<true>(r, voff + (uint32_t)k * rsb); }
  __device__ __forceinline__ void store(__amdgpu_buffer_rsrc_t r, int k, i32x4 v) const { buf_st16<true>(r, voff + (uint32_t)k * rsb, v); }
};
template <typename TI, int V> __device__ __forceinline__ void glr_cvt(i32x4 r, float (&v)[V]) {
  typedef TI vec __attribute__((ext_vector_type(V)));
  const vec b = __builtin_bit_cast(vec, r);
#pragma unroll
  for (int j = 0; j < V; ++j) v[j] = (float)b[j];
}
template <typename TI, int V> __device__ __forceinline__ i32x4 glr_raw(const float (&v)[V]) {
  typedef TI vec __attribute__((ext_vector_type(V)));
  vec b;
#pragma unroll
  for (int j = 0; j < V; ++j) b[j] = (TI)v[j];
  return __builtin_bit_cast(i32x4, b);
}

// rate softplus(lambda), kept finite (an infinite exponent times a state would be NaN where a is zero).
__device__ __forceinline__ float glr_rate(float rate, float lam) {
  const float c = rate * softplusf(lam);
  return c > 0x1p100f ? 0x1p100f : c;
}

// The sigmoid. Of float32 rows: exp(-z) = 2^(t + lo), the product with log2(e) in two parts, the hardware's power (1 ulp), and its
// reciprocal with a Newton step, together 3 ulp; below -87 zero (float32 keeps no more there), past 87 one. With expf and a division
// a prompt of 8192 x 4096 took 170 us, so 145.
template <typename TI> __device__ __forceinline__ float glr_sigmoid(float z) {
  if constexpr (sizeof(TI) == 2) {
    return sigmoidf<TI>(z);
  } else {
    const bool gone = z < -87.f;
    z = gone ? -87.f : z;  // (a NaN stays)
    z = z > 87.f ? 87.f : z;
    const float t = z * -1.44269504f, lo = fmaf(z, -1.92596299e-8f, fmaf(z, -1.44269504f, -t));
    const float x = __builtin_amdgcn_exp2f(t), d = fmaf(x, lo * 0.693147181f, x) + 1.f;
    const float r = __builtin_amdgcn_rcpf(d);
    return gone ? 0.f : fmaf(fmaf(-d, r, 1.f), r, r);
  }
}

// s(z) and its complement 1 - s(z) = s(-z) of float32 rows, as in glr_sigmoid from x = exp(-|z|): 1 / (1 + x) and x / (1 + x). (One minus
// the rounded s keeps 2^-24 of one: at z = 12 1% of itself is wrong, at 17 all.)
__device__ __forceinline__ void glr_sides(float z, float& s, float& c) {
  const bool gone = fabsf(z) > 87.f;
  const float y = gone ? 87.f : fabsf(z);  // (a NaN stays)
  const float t = y * -1.44269504f, lo = fmaf(y, -1.92596299e-8f, fmaf(y, -1.44269504f, -t));
  const float p = __builtin_amdgcn_exp2f(t), x = fmaf(p, lo * 0.693147181f, p), d = x + 1.f;
  const float r = __builtin_amdgcn_rcpf(d), big = fmaf(fmaf(-d, r, 1.f), r, r), small = gone ? 0.f : x * big;
  s = z > 0.f ? big : small;
  c = z > 0.f ? small : big;
}
// Whether some gate of a wave's bfloat16 rows is past 7 (or a NaN), from where on 1 - s of the rounded s is more than 2e-4 of itself off.
template <int K> __device__ __forceinline__ bool glr_open(const i32x4 (&r)[K], const i32x4 (&i)[K]) {
  typedef short s16x2 __attribute__((ext_vector_type(2)));
  s16x2 m{0, 0};  // (positive values are ordered as their bits are, negative ones below zero)
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int j = 0; j < 4; ++j)
      m = __builtin_elementwise_max(m, __builtin_elementwise_max(__builtin_bit_cast(s16x2, r[k][j]), __builtin_bit_cast(s16x2, i[k][j])));
  return __any((m[0] > m[1] ? m[0] : m[1]) > 0x40E0);
}

// exp(-L), for L >= 0.
template <typename TI> __device__ __forceinline__ float glr_exp(float L) {
  if constexpr (sizeof(TI) == 2) return __builtin_amdgcn_exp2f(L * -1.44269504f);
  else return expf(-L);
}
// 1 - exp(-L): below a quarter L q(L) with q of degree 4 through (1 - exp(-L)) / L at the five Chebyshev points of
// [0, 1/4] (5e-9 off). `deep` (wave-uniform): some L may be more; where no channel's rate is, the exponentials are left out.
template <typename TI, int V> __device__ __forceinline__ void one_minus_exp(const float (&L)[V], bool deep, float (&e)[V]) {
#pragma unroll
  for (int j = 0; j < V; ++j) {
    float q = fmaf(L[j], 0.007513606f, -0.041490655f);
    q = fmaf(L[j], q, 0.166651085f);
    q = fmaf(L[j], q, -0.49999952f);
    q = fmaf(L[j], q, 1.f);
    e[j] = L[j] * q;
  }
  if (deep) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      float x = L[j];
      asm volatile("" : "+v"(x));  // (keeps the branch: not eight exponentials for nothing)
      e[j] = x < 0.25f ? e[j] : 1.f - glr_exp<TI>(x);
    }
  }
}

// w = sqrt(1 - a^2) = sqrt(e (1 + a)) of e and a1 = 1 - e, by the hardware's root (1 ulp), and 1 / w, which ends at 2^63 (L / w
// is then zero where L is). A w below 2^-63, whose square no float32 holds in full, may come out as less.
__device__ __forceinline__ float glr_weight(float e, float a1) { return __builtin_amdgcn_sqrtf(fmaf(e, a1, e)); }
__device__ __forceinline__ float glr_inv_weight(float e, float a1) { return __builtin_amdgcn_rsqf(fmaxf(fmaf(e, a1, e), 0x1p-126f)); }

// x of the lane that CTRL names, zero where it lies outside the row of 16 (e = 0, b = 0: the map that changes nothing).
template <int CTRL> __device__ __forceinline__ float dpp_or0(float x) {
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), CTRL, 0xF, 0xF, true));
}
// (E, B) <- first (E1, B1), then (E, B): with A = 1 - E, E + E1 A and B + B1 A. E1 A is rounded relative to itself, so a sum of
// small E keeps its bits.
__device__ __forceinline__ void glr_after(float E1, float B1, float& E, float& B) {
  const float A = 1.f - E;
  E = fmaf(E1, A, E);
  B = fmaf(B1, A, B);
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

// How a launch cuts its sequences: one of at most `keep` tokens is a segment, a longer one is cut into segments of `seg`
// (a multiple of a tile; `per` of them to a sequence where there is no table).
struct GlrPlan {
  int seg, keep, per, slots, blocks;  // segment slots, channel blocks
  bool cut;                           // some sequence may have more than one segment
};

// Segment `slot` of the launch: tokens [t0, t1), the k-th of sequence n's `segs` (rows [lo, hi)). The slots of a packed batch
// of up to kGlrEven sequences are its segments, one after the other; of a larger one segment k has slot lo / seg + n + k, below
// T_total / seg + N, and some are empty. (Empty workgroups among the others make the dispatcher put two of these on one
// compute unit: 4 x 4096 x 2560 took 160 us instead of 97.)
constexpr int kGlrEven = 256;
struct GlrSeg {
  int n, k, segs;
  int64_t lo, hi, t0, t1;
};
__device__ __forceinline__ int glr_size(const GlrPlan& p, int len) { return len <= p.keep ? p.keep : p.seg; }
__device__ __forceinline__ int glr_segs(const GlrPlan& p, int len) {
  const int size = glr_size(p, len);
  return len <= size ? 1 : (len + size - 1) / size;
}
__device__ __forceinline__ bool glr_seg(const GlrArgs& a, const GlrPlan& p, int slot, GlrSeg& q) {
  auto rows = [&](int n, int64_t& lo, int64_t& hi) {  // of a packed sequence, clamped into the caller's
    const int64_t x = a.cu[n], y = a.cu[n + 1];
    lo = x < 0 ? 0 : x > a.rows ? a.rows : x;
    hi = y < lo ? lo : y > a.rows ? a.rows : y;
  };
  if (!a.cu) {
    q.n = slot / p.per;
    q.k = slot - q.n * p.per;
    q.lo = (int64_t)q.n * a.T;
    q.hi = q.lo + a.T;
  } else if (a.N <= kGlrEven) {
    constexpr int U = kGlrEven / 64;  // lane l looks at sequences U l .. U l + U - 1
    int cnt[U], sum = 0;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      cnt[u] = 0;
      if (lane_id() * U + u < a.N) {
        int64_t lo, hi;
        rows(lane_id() * U + u, lo, hi);
        cnt[u] = glr_segs(p, (int)(hi - lo));
      }
      sum += cnt[u];
    }
    int at = wave_scan_incl_int(sum) - sum, n = -1, k = 0;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (slot >= at && slot < at + cnt[u]) {
        n = lane_id() * U + u;
        k = slot - at;
      }
      at += cnt[u];
    }
    const uint64_t who = __ballot(n >= 0);
    if (who == 0) return false;
    const int l = __builtin_ctzll(who);
    q.n = __builtin_amdgcn_readlane(n, l);
    q.k = __builtin_amdgcn_readlane(k, l);
    rows(q.n, q.lo, q.hi);
  } else {
    int l = 0;
    for (int n = a.N; n > 1;) {  // the largest n whose first slot is at most `slot`, 64 probes at a time
      const int stride = (n + 63) / 64, i = lane_id() * stride;
      int64_t lo, hi;
      rows(l + (i < n ? i : 0), lo, hi);
      const uint64_t m = __ballot(i < n && (int)((uint32_t)lo / (uint32_t)p.seg) + l + i <= slot);
      const int at = (m ? 63 - __builtin_clzll(m) : 0) * stride;
      l += at;
      n = n - at < stride ? n - at : stride;
    }
    q.n = __builtin_amdgcn_readfirstlane(l);
    rows(q.n, q.lo, q.hi);
    q.k = slot - (int)((uint32_t)q.lo / (uint32_t)p.seg) - q.n;
  }
  const int len = (int)(q.hi - q.lo), size = glr_size(p, len);
  q.segs = glr_segs(p, len);
  if (q.k < 0 || q.k >= q.segs) return false;
  q.t0 = q.lo + (int64_t)q.k * size;
  q.t1 = q.t0 + size < q.hi ? q.t0 + size : q.hi;
  return true;
}

// Workgroup -> (segment slot, first channel): channel blocks run fastest, so that workgroups in flight read whole rows.
#define GLR_PLACE                                                                        \
  constexpr int V = glr_v<TI>(), CB = 8 * V;                                             \
  const int slot = (int)blockIdx.x / pl.blocks, c0 = ((int)blockIdx.x - slot * pl.blocks) * CB; \
  const GlrLane me;                                                                      \
  const bool on = c0 + me.cg * V < a.ch;                                                 \
  const int c = on ? c0 + me.cg * V : 0, ci = c0 + lane_id();                            \
  const bool mine = lane_id() < CB && ci < a.ch; /* a channel of the scanning waves */   \
  const int cl = c0 + lane_id() % CB;                                                    \
  const float lam = a.lam[cl < a.ch ? cl : a.ch - 1]
// Rates of a thread's channels, each found by one lane of the wave; a lane of no channel has that of the last.
#define GLR_RATES                                                                        \
  const float its = glr_rate(a.rate, lam);                                               \
  float rate[V];                                                                         \
  _Pragma("unroll") for (int j = 0; j < V; ++j) rate[j] = __shfl(its, me.cg * V + j);    \
  const bool deep = __any(!(its < 0.25f))

// ------------------------------------------------------------------ maps of segments
// The map of each segment that another one continues from: forward every one but a sequence's last, backward
// every one but its first. A thread row takes a contiguous run of the tokens. [slot][E | B][ch].
template <typename TI, bool FWD> __global__ __launch_bounds__(GNT) void k_glr_map(GlrArgs a, GlrPlan pl) {
  GlrSeg q;
  GLR_PLACE;
  __shared__ float sE[GE][CB], sB[GE][CB];
  if (!glr_seg(a, pl, slot, q) || (FWD ? q.k == q.segs - 1 : q.k == 0)) return;
  GLR_RATES;
  // a thread row's run of the tokens, one of them ahead in flight (four took more registers, and then half the waves:
  // 16384 x 4096 tokens 94 us, with one 83)
  const int run = (int)((q.t1 - q.t0 + GROWS - 1) / GROWS);
  const bool fresh = FWD && a.fresh && q.k == 0 && a.fresh[q.n] != 0;
  float E[V], B[V];
#pragma unroll
  for (int j = 0; j < V; ++j) E[j] = B[j] = 0.f;
  const int64_t begin = q.t0 + (int64_t)me.tt * run;
  const TI *pr = static_cast<const TI*>(a.r) + c, *px = static_cast<const TI*>(FWD ? a.x : a.dy) + c, *pi = static_cast<const TI*>(a.i) + c;
  const int64_t x_rs = FWD ? a.x_rs : a.dy_rs;
  i32x4 rr, rx, ri;
  auto load = [&](int64_t t) {
    const int64_t row = t < q.t1 ? t : q.t1 - 1;
    rr = *reinterpret_cast<const i32x4*>(pr + row * a.r_rs);
    rx = *reinterpret_cast<const i32x4*>(px + row * x_rs);
    if constexpr (FWD) ri = *reinterpret_cast<const i32x4*>(pi + row * a.i_rs);
  };
  load(FWD ? begin : begin + run - 1);
  for (int b = 0; b < run; ++b) {
    const int64_t t = FWD ? begin + b : begin + run - 1 - b;
    float r[V], x[V], iv[V], L[V], e[V];
    glr_cvt<TI, V>(rr, r);
    glr_cvt<TI, V>(rx, x);
    if constexpr (FWD) glr_cvt<TI, V>(ri, iv);
    if (b + 1 < run) load(FWD ? t + 1 : t - 1);
    if (t >= q.t1) continue;
#pragma unroll
    for (int j = 0; j < V; ++j) L[j] = rate[j] * glr_sigmoid<TI>(r[j]);
    one_minus_exp<TI, V>(L, deep, e);
    if (fresh && t == q.lo)
#pragma unroll
      for (int j = 0; j < V; ++j) e[j] = 1.f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const float a1 = 1.f - e[j];
      if constexpr (FWD) B[j] = fmaf(a1, B[j], glr_weight(e[j], a1) * (glr_sigmoid<TI>(iv[j]) * x[j]));
      else B[j] = a1 * (B[j] + x[j]);
      E[j] = fmaf(E[j], a1, e[j]);
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

// h through the maps of `count` segments, the first at m, the others behind it (dir 1) or in front (-1); sixteen of them under way
// at once (one after the other took 0.25 us each: a prompt of 131072 x 64, in 512 segments, 147 us, so 42, by eights 50).
constexpr int GF = 16;
__device__ __forceinline__ float glr_fold(const float* m, int ch, int dir, int count, float h) {
  const int64_t step = (int64_t)dir * 2 * ch;
  for (int s = 0; s < count; s += GF) {
    float e[GF], b[GF];
#pragma unroll
    for (int i = 0; i < GF; ++i) {
      const float* p = m + (s + i < count ? s + i : s) * step;
      e[i] = p[0];
      b[i] = p[ch];
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < GF; ++i) h = s + i < count ? fmaf(-e[i], h, h) + b[i] : h;
  }
  return h;
}

// ------------------------------------------------------------------ forward
template <typename TI, bool SAVE> __global__ __launch_bounds__(GNT) void k_glr_fwd(GlrArgs a, GlrPlan pl) {
  GlrSeg q;
  GLR_PLACE;
  __shared__ float sE[GE][CB], sB[GE][CB], sh[GE][CB];
  if (!glr_seg(a, pl, slot, q)) return;
  const GlrView<TI> vx(a.x, a.x_rs, on, me.tt * GK, c), vr(a.r, a.r_rs, on, me.tt * GK, c), vi(a.i, a.i_rs, on, me.tt * GK, c),
      vy(a.y, a.y_rs, on, me.tt * GK, c);
  auto left = [&](int64_t t) { return (int)(q.t1 - t < GTILE ? q.t1 - t : GTILE); };
  i32x4 rx[GK], rr[GK], ri[GK];
  auto load = [&](int64_t t) {
    const int n = left(t);
    const auto sr = vr.rows(t, n), si = vi.rows(t, n), sx = vx.rows(t, n);
#pragma unroll
    for (int k = 0; k < GK; ++k) {
      rr[k] = vr.load(sr, k);
      ri[k] = vi.load(si, k);
      rx[k] = vx.load(sx, k);
    }
  };
  if (q.t0 < q.t1) load(q.t0);
  GLR_RATES;
  const bool fresh = a.fresh && a.fresh[q.n] != 0;
  float h = 0.f;  // wave 0: the carried state of channel ci
  if (wave_id() == 0 && mine) {
    h = fresh || !a.h0 ? 0.f : a.h0[(int64_t)q.n * a.ch + ci];
    h = glr_fold(a.ws + (int64_t)(slot - q.k) * 2 * a.ch + ci, a.ch, 1, q.k, h);
  }
  for (int64_t t = q.t0; t < q.t1; t += GTILE) {
    float a1[GK][V], b[GK][V], E[V], B[V], Ex[V], Bx[V];  // a1 = 1 - e: what a map does to the tokens of this thread alone
    const bool plain = t + GTILE <= q.t1 && !(fresh && t == q.lo);
#pragma unroll
    for (int k = 0; k < GK; ++k) {
      float x[V], r[V], i[V], L[V], e[V];
      glr_cvt<TI, V>(rx[k], x);
      glr_cvt<TI, V>(rr[k], r);
      glr_cvt<TI, V>(ri[k], i);
#pragma unroll
      for (int j = 0; j < V; ++j) L[j] = rate[j] * glr_sigmoid<TI>(r[j]);
      one_minus_exp<TI, V>(L, deep, e);
      if (!plain) {
        const int64_t row = t + me.tt * GK + k;
        if (fresh && row == q.lo)
#pragma unroll
          for (int j = 0; j < V; ++j) e[j] = 1.f;
        if (row >= q.t1)  // a token that changes nothing
#pragma unroll
          for (int j = 0; j < V; ++j) e[j] = x[j] = 0.f;
      }
#pragma unroll
      for (int j = 0; j < V; ++j) {
        a1[k][j] = 1.f - e[j];
        b[k][j] = glr_weight(e[j], a1[k][j]) * (glr_sigmoid<TI>(i[j]) * x[j]);
        B[j] = k ? fmaf(a1[k][j], B[j], b[k][j]) : b[k][j];
        E[j] = k ? fmaf(E[j], a1[k][j], e[j]) : e[j];
      }
    }
    if (t + GTILE < q.t1) load(t + GTILE);
    glr_scan4<true, V>(E, B, Ex, Bx);
    if (me.last)
#pragma unroll
      for (int j = 0; j < V; ++j) {
        sE[me.g][me.cg * V + j] = E[j];
        sB[me.g][me.cg * V + j] = B[j];
      }
    lds_barrier();
    if (wave_id() == 0 && lane_id() < CB) {
      if (SAVE && mine) a.sv[(q.lo / GTILE + q.n + (t - q.lo) / GTILE) * a.ch + ci] = h;
#pragma unroll
      for (int g = 0; g < GE; ++g) {
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
    for (int k = 0; k < GK; ++k) {
#pragma unroll
      for (int j = 0; j < V; ++j) y[j] = fmaf(a1[k][j], y[j], b[k][j]);
      vy.store(out, k, glr_raw<TI, V>(y));
    }
  }
  if (a.hT && wave_id() == 0 && mine && q.k == q.segs - 1) a.hT[(int64_t)q.n * a.ch + ci] = h;
}

// ------------------------------------------------------------------ backward
// Tiles from the last to the first; within a tile the states from its saved start and the gradients from
// those behind it side by side. Partials of dlambda: [slot][ch].
template <typename TI> __global__ __launch_bounds__(GNT) void k_glr_bwd(GlrArgs a, GlrPlan pl, float* part) {
  GlrSeg q;
  GLR_PLACE;
  __shared__ float sE[GE][CB], sB[GE][CB], sC[GE][CB], sh[GE][CB], sg[GE][CB];
  __shared__ i32x4 raw[sizeof(TI) == 2 ? 2 * GK : 1][GNT];
  if (!glr_seg(a, pl, slot, q)) {
    if (part && wave_id() == 0 && mine) part[(int64_t)slot * a.ch + ci] = 0.f;
    return;
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
      rr[k] = vr.load(sr, k);
      ri[k] = vi.load(si, k);
      rx[k] = vx.load(sx, k);
      rd[k] = vd.load(sd, k);
    }
  };
  const int64_t tiles = (q.t1 - q.t0 + GTILE - 1) / GTILE;
  if (tiles) load(q.t0 + (tiles - 1) * GTILE);
  GLR_RATES;
  const bool fresh = a.fresh && a.fresh[q.n] != 0;
  float cc = 0.f;  // wave 1: the gradient that flows into the tile's end
  if (wave_id() == 1 && mine) {
    cc = a.dhT ? a.dhT[(int64_t)q.n * a.ch + ci] : 0.f;
    int last = slot - q.k + q.segs - 1;  // (of sequences that overlap, in a malformed table, more than the slots hold)
    if (last >= pl.slots) last = pl.slots - 1;
    cc = glr_fold(a.ws + (int64_t)last * 2 * a.ch + ci, a.ch, -1, last - slot, cc);
  }
  float dl[V];
#pragma unroll
  for (int j = 0; j < V; ++j) dl[j] = 0.f;
  for (int64_t tile = tiles - 1; tile >= 0; --tile) {
    const int64_t t = q.t0 + tile * GTILE;
    float hs = 0.f;  // wave 0: the tile's saved start
    if (wave_id() == 0 && mine) hs = a.sv[((q.lo / GTILE) + q.n + (t - q.lo) / GTILE) * a.ch + ci];
    const bool plain = t + GTILE <= q.t1 && !(fresh && t == q.lo);
    // The gates' complements. For those of bfloat16 rows there are not registers enough: they are formed at their use, as 1 - s, and where
    // a gate is too open for that from its rows, kept in LDS. (4 x 4096 x 2560 176 us, without complements 170, with s(-|z|) under the
    // sign of z in the place of s 188; gates past 7 in every tile take 30 more.)
    float cr[GK][V], ci[GK][V];
    float e[GK][V], sr[GK][V], si[GK][V], rw[GK][V], E[V], B[V], Ex[V], Bx[V], F[V], C[V], Fx[V], Cx[V];
    i32x4 kx[GK], kd[GK];
    bool open = false;
    if constexpr (sizeof(TI) == 2) open = glr_open(rr, ri);
    if (open)  // (read by the thread that writes it)
#pragma unroll
      for (int k = 0; k < GK; ++k) {
        raw[2 * k][threadIdx.x] = rr[k];
        raw[2 * k + 1][threadIdx.x] = ri[k];
      }
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
        if constexpr (sizeof(TI) == 2) {
          sr[k][j] = glr_sigmoid<TI>(r[j]);
          si[k][j] = glr_sigmoid<TI>(i[j]);
        } else {
          glr_sides(r[j], sr[k][j], cr[k][j]);
          glr_sides(i[j], si[k][j], ci[k][j]);
        }
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
        const float a1 = 1.f - e[k][j];
        rw[k][j] = glr_inv_weight(e[k][j], a1);
        const float b = fmaf(e[k][j], a1, e[k][j]) * rw[k][j] * (si[k][j] * x[j]);
        B[j] = k ? fmaf(a1, B[j], b) : b;
        E[j] = k ? fmaf(E[j], a1, e[k][j]) : e[k][j];
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
      for (int j = 0; j < V; ++j) asm volatile("" : "+v"(e[k][j]), "+v"(sr[k][j]), "+v"(si[k][j]), "+v"(rw[k][j]));
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
        hp[k + 1][j] = fmaf(1.f - e[k][j], hp[k][j], fmaf(e[k][j], 1.f - e[k][j], e[k][j]) * rw[k][j] * (si[k][j] * x[j]));
    }
    const auto tx = ox.rows(t, left(t)), tr = orr.rows(t, left(t)), ti = oi.rows(t, left(t));
#pragma unroll
    for (int k = GK - 1; k >= 0; --k) {
      const int64_t row = t + me.tt * GK + k;
      float x[V], d[V], dx[V], dr[V], di[V];
      glr_cvt<TI, V>(kx[k], x);
      glr_cvt<TI, V>(kd[k], d);
      if constexpr (sizeof(TI) == 2) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
          cr[k][j] = 1.f - sr[k][j];
          ci[k][j] = 1.f - si[k][j];
        }
        if (open) {
          float r[V], i[V];
          glr_cvt<TI, V>(raw[2 * k][threadIdx.x], r);
          glr_cvt<TI, V>(raw[2 * k + 1][threadIdx.x], i);
#pragma unroll
          for (int j = 0; j < V; ++j) {
            cr[k][j] = glr_sigmoid<TI>(-r[j]);
            ci[k][j] = glr_sigmoid<TI>(-i[j]);
          }
        }
      }
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float G = cg[j] + d[j], u = si[k][j] * x[j], L = rate[j] * sr[k][j], a1 = 1.f - e[k][j];
        float al = a1;  // a to its own last bits
        if (deep && !(fresh && row == q.lo)) {
          float y = L;
          asm volatile("" : "+v"(y));
          al = y < 0.25f ? a1 : glr_exp<TI>(y);
        }
        const float du = fmaf(e[k][j], a1, e[k][j]) * rw[k][j] * G;
        dx[j] = si[k][j] * du;
        di[j] = u * ci[k][j] * du;
        // L dL; a and L first, whose product stays finite
        const float LdL = (al * L) * G * fmaf(u * al, rw[k][j], -hp[k][j]);
        dr[j] = LdL * cr[k][j];
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
      // sigmoid / softplus: one to float32 below -20 (and expf(-lam) ends at -88, where softplus does not); where softplus is zero, so
      // are the exponents
      const float q = lam < -20.f ? 1.f : 1.f / (1.f + expf(-lam)) / sp;
      part[(int64_t)slot * a.ch + ci] = sp > 0.f ? s * q : 0.f;
    }
  }
}

// ------------------------------------------------------------------ one token
// Two channels per thread: softplus takes some 100 instructions, and the calls are short (one row of 2560 2.9 us, 256 rows 5.0; with
// eight channels 4.8 and 6.8). Many rows are bound by HBM either way: 4096 x 4096 60 and 58 us.
constexpr int GD = kGlrTokenChannels / 64;
template <typename TI> __global__ __launch_bounds__(64) void k_glr_decode(GlrArgs a) {
  typedef TI vec __attribute__((ext_vector_type(GD)));
  typedef float fvec __attribute__((ext_vector_type(GD)));
  const int c = (int)(blockIdx.y * 64 + threadIdx.x) * GD, n = (int)blockIdx.x;
  if (c >= a.ch) return;
  const int slot = a.idx ? a.idx[n] : n;
  if (slot < 0 || slot >= a.n_slots) return;
  const bool fresh = a.fresh && a.fresh[n] != 0;
  fvec* st = reinterpret_cast<fvec*>(a.state + (int64_t)slot * a.ch + c);
  const vec x = *reinterpret_cast<const vec*>((const TI*)a.x + (int64_t)n * a.x_rs + c);
  const vec r = *reinterpret_cast<const vec*>((const TI*)a.r + (int64_t)n * a.r_rs + c);
  const vec i = *reinterpret_cast<const vec*>((const TI*)a.i + (int64_t)n * a.i_rs + c);
  const fvec lam = *reinterpret_cast<const fvec*>(a.lam + c);
  fvec h = fvec{};
  if (!fresh) h = *st;
  float L[GD], e[GD];
#pragma unroll
  for (int j = 0; j < GD; ++j) L[j] = glr_rate(a.rate, lam[j]) * glr_sigmoid<TI>((float)r[j]);
  one_minus_exp<TI, GD>(L, true, e);
  vec y;
#pragma unroll
  for (int j = 0; j < GD; ++j) {
    const float u = glr_sigmoid<TI>((float)i[j]) * (float)x[j];
    h[j] = fresh ? u : fmaf(-e[j], h[j], h[j]) + glr_weight(e[j], 1.f - e[j]) * u;
    y[j] = (TI)h[j];
  }
  *st = h;
  *reinterpret_cast<vec*>((TI*)a.y + (int64_t)n * a.y_rs + c) = y;
}

// ------------------------------------------------------------------ launches
// A workgroup that walks down its sequence reads everything once, but a single chain takes 2.7 us a tile (gates of 2 x
// 64 x 64 values in eight waves, half of it exponentials, reciprocals and roots): 16384 tokens x 4096 channels by 64
// workgroups 331 us, cut into eighths by 512 169 with the pass for their maps; 4 x 4096 x 2560 by 160 workgroups 95 us, cut
// into quarters 80 + 75. So a sequence is cut, finely, where it is longer than its share of 128 workgroups, down to two tiles
// (a training step of 1024 x 2560, whole 73 us, by two tiles 51; of 3800 float32 tokens x 512, by two tiles 43, by one 50) but
// not up to 512 tokens (500 and 300 tokens x 2560 44 us, with 256 for 512 42, one prompt of 300 x 1024 12.8 and 17.7). On either side of the
// 128 (training steps of sequences of 4096 x 2560): three are cut, 216 us, whole 267; four are not, 282, cut 288; five 302 and 382.
static GlrPlan glr_plan(const GlrArgs& a, int dtype) {
  GlrPlan p;
  const int CB = dtype == 0 ? 32 : 64;
  p.blocks = (a.ch + CB - 1) / CB;
  const int64_t longest = a.cu ? a.rows : a.T, work = a.rows * p.blocks;
  auto tiles = [](int64_t t, int64_t least) {  // (a batch has up to 2^28 tokens)
    return ((t < least ? least : t < 1 << 28 ? t : 1 << 28) + GTILE - 1) / GTILE * GTILE;
  };
  p.keep = (int)tiles(work / 128, 512);
  p.seg = (int)tiles(work / 512, 256);
  p.cut = longest > p.keep;
  if (!p.cut) p.seg = p.keep;
  p.per = a.cu ? 0 : p.cut ? (int)((a.T + p.seg - 1) / p.seg) : 1;
  p.slots = a.cu ? (int)(a.rows / p.seg) + a.N : a.N * p.per;
  return p;
}
int64_t glr_blocks(const GlrArgs& a, int dtype) {
  const GlrPlan p = glr_plan(a, dtype);
  return (int64_t)p.slots * p.blocks;
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
  const unsigned grid = (unsigned)p.slots * (unsigned)p.blocks;
  if (grid == 0) return hipSuccess;
  if (p.cut) {
    traced("k_glr_map", s, [&] { k_glr_map<TI, true><<<grid, GNT, 0, s>>>(a, p); });
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  traced("k_glr_fwd", s, [&] {
    if (a.sv) k_glr_fwd<TI, true><<<grid, GNT, 0, s>>>(a, p);
    else k_glr_fwd<TI, false><<<grid, GNT, 0, s>>>(a, p);
  });
  return hipGetLastError();
}

template <typename TI> static hipError_t glr_backward(const GlrArgs& a, int dtype, hipStream_t s) {
  const GlrPlan p = glr_plan(a, dtype);
  const unsigned grid = (unsigned)p.slots * (unsigned)p.blocks;
  hipError_t e = hipSuccess;
  if (p.cut && grid) {
    traced("k_glr_map", s, [&] { k_glr_map<TI, false><<<grid, GNT, 0, s>>>(a, p); });
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  float* part = a.dlam ? a.ws + (p.cut ? (int64_t)p.slots * 2 * a.ch : 0) : nullptr;
  if (grid) traced("k_glr_bwd", s, [&] { k_glr_bwd<TI><<<grid, GNT, 0, s>>>(a, p, part); });
  e = hipGetLastError();
  if (e == hipSuccess && a.dlam) e = launch_colsum(part, p.slots, a.ch, ColsumOut{{a.dlam, nullptr, nullptr}}, 1, s);
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
  const dim3 grid((unsigned)a.N, (unsigned)((a.ch + kGlrTokenChannels - 1) / kGlrTokenChannels));
  traced("k_glr_decode", s, [&] {
    if (dtype == 0) k_glr_decode<float><<<grid, 64, 0, s>>>(a);
    else k_glr_decode<__bf16><<<grid, 64, 0, s>>>(a);
  });
  return hipGetLastError();
}

}  // namespace gdn
