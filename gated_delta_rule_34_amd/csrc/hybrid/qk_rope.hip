// qk_rope.hip -- RMS norm of each query and key head with the rotation of its position, on gfx950:
// forward, gradients, and the serving form that writes keys and values into the pages of a cache.
//
//   n = v rs w,  rs = 1 / sqrt(mean(v^2) + eps);  pairs (a, b) of n: (a cos - b sin, a sin + b cos) scale
//   backward: t = dy turned back (times scale), dw = sum t v rs,  dv = rs (t w - n' mean(t w n')) of n' = v rs
//
// Streaming work: every head is read and written once, bound by HBM. LH lanes hold a head, eight
// adjacent values each; a pair's other half is the same lane's (adjacent pairs) or comes from the lane rot / 16 away. A
// workgroup takes a few rows: the angles of a row serve all its heads, so each is found once, by one thread, and
// kept in LDS. Angles are float64 products reduced to an eighth of a turn in float64; only then do sine and
// cosine follow, from their series in float32.
#include "../gdn_common.h"
#include "../layer/vec8.h"
#include "hybrid_internal.h"

namespace gdn {

constexpr int RNT = 256;
constexpr int RROWS = 2;  // rows of a workgroup at the most

// (cos, sin) of the angle pos f, times scale. The quarter turn that is nearest leaves at most pi / 4, whose series
// end with z^5 (2e-8 of the sum).
__device__ __forceinline__ float2 rope_angle(int pos, double f, float scale) {
  const double y = (double)pos * f * 0.63661977236758134308, k = rint(y);
  const float t = (float)((y - k) * 1.57079632679489661923), z = t * t;
  const int quad = (int)(k - 4.0 * floor(k * 0.25));
  float s = fmaf(z, 1.f / 362880.f, -1.f / 5040.f);
  s = fmaf(z, s, 1.f / 120.f);
  s = fmaf(z, s, -1.f / 6.f);
  s = fmaf(t * z, s, t);
  float c = fmaf(z, -1.f / 3628800.f, 1.f / 40320.f);
  c = fmaf(z, c, -1.f / 720.f);
  c = fmaf(z, c, 1.f / 24.f);
  c = fmaf(z, c, -0.5f);
  c = fmaf(z, c, 1.f);
  const float cc = quad & 1 ? s : c, ss = quad & 1 ? c : s;
  return float2{(quad == 1 || quad == 2 ? -cc : cc) * scale, (quad >= 2 ? -ss : ss) * scale};
}

// Sum over the LH lanes of a head, in each of them.
template <int LH> __device__ __forceinline__ float head_sum(float x) {
  x += dpp<0xB1>(x);   // quad_perm [1, 0, 3, 2]
  x += dpp<0x4E>(x);   // quad_perm [2, 3, 0, 1]
  if constexpr (LH >= 8) x += dpp<0x141>(x);   // row_half_mirror
  if constexpr (LH >= 16) x += dpp<0x140>(x);  // row_mirror
  if constexpr (LH >= 32) x += __shfl_xor(x, 16);
  return x;
}

// The piece of eight values that the lane `d` away holds.
template <typename TI> __device__ __forceinline__ Raw8<TI> lane_away(const Raw8<TI>& x, int d) {
  Raw8<TI> y;
  const int at = (lane_id() + d) << 2;
  if constexpr (sizeof(TI) == 2) {
#pragma unroll
    for (int j = 0; j < 4; ++j) y.a[j] = __builtin_amdgcn_ds_bpermute(at, x.a[j]);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      y.a[j] = __int_as_float(__builtin_amdgcn_ds_bpermute(at, __float_as_int(x.a[j])));
      y.b[j] = __int_as_float(__builtin_amdgcn_ds_bpermute(at, __float_as_int(x.b[j])));
    }
  }
  return y;
}

// A lane's place in its head: its values [c, c + 8); whether they are rotated; the distance to the lane with
// their pairs' other halves (0: they are its own); the first of their angles; the sign of the sine.
struct RopePlace {
  int li, c, away, ang;
  bool live, turned;
  float sign;
  __device__ __forceinline__ RopePlace(int LH, int D, int R, bool adjacent) {
    li = (int)threadIdx.x % LH;
    c = li * 8;
    live = c < D;
    turned = c < R;
    const int half = R / 16;
    const bool low = li < half;
    away = !turned || adjacent ? 0 : low ? half : -half;
    ang = adjacent ? li * 4 : (low ? li : li - half) * 8;
    sign = low ? -1.f : 1.f;
  }
};

// Angles of the workgroup's rows: cs[row][rot / 2].
__device__ __forceinline__ void rope_angles(const RopeArgs& a, int64_t row0, int nrows, float2* cs) {
  const int half = a.R / 2;
  for (int q = (int)threadIdx.x; q < nrows * half; q += RNT) {
    const int row = q / half;
    cs[q] = rope_angle(a.pos[row0 + row], a.freq[q - row * half], a.scale);
  }
}

__device__ __forceinline__ F8 rope_weight(const float* w, int c, bool live) {
  if (w && live) return ld8<float>(w + c);
  return F8{{1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f}};
}

// The item's heads: queries, then keys, then (cache form) values. Both forms give the same bits: what is fused is
// written out.
template <typename TI, int LH, bool ADJ, bool CACHE> __global__ __launch_bounds__(RNT) void k_rope_fwd(RopeArgs a, int rb) {
#pragma clang fp contract(off)
  __shared__ float2 cs[RROWS * 128];
  __shared__ int64_t rows_at[RROWS];  // of a row's first key head among the pool's rows, or -1: not cached
  const RopePlace me(LH, a.D, a.R, ADJ);
  const int64_t row0 = (int64_t)blockIdx.x * rb;
  const int nrows = (int)(a.rows - row0 < rb ? a.rows - row0 : rb);
  const int H = a.Hq + a.Hk * (CACHE ? 2 : 1), items = nrows * H;
  constexpr int SLOTS = RNT / LH;
  auto source = [&](int it) {
    const int row = it / H, h = it - row * H;
    const int64_t t = row0 + row;
    const TI* p = h < a.Hq ? (const TI*)a.q + t * a.q_rs + h * a.D
                  : !CACHE || h < a.Hq + a.Hk ? (const TI*)a.k + t * a.k_rs + (h - a.Hq) * a.D
                                              : (const TI*)a.v + t * a.v_rs + (h - a.Hq - a.Hk) * a.D;
    return ldraw8<true, TI>(p + (me.live ? me.c : 0));
  };
  int it = (int)threadIdx.x / LH;
  Raw8<TI> next;
  if (it < items) next = source(it);
  const F8 wq = rope_weight(a.wq, me.c, me.live), wk = rope_weight(a.wk, me.c, me.live);
  F8 oq, ok;  // the weights of the pairs' other halves
  if constexpr (!ADJ) {
    oq = rope_weight(a.wq, me.c + me.away * 8, me.live);
    ok = rope_weight(a.wk, me.c + me.away * 8, me.live);
  }
  if (CACHE && (int)threadIdx.x < nrows) {
    const int64_t w = a.where[row0 + threadIdx.x];
    const uint32_t page = (uint32_t)w / (uint32_t)a.page;
    rows_at[threadIdx.x] = w < 0 || w >= a.places ? -1 : (int64_t)page * a.Hk * a.page + (w - (int64_t)page * a.page);
  }
  rope_angles(a, row0, nrows, cs);
  __syncthreads();
  for (; it < items; it += SLOTS) {
    const Raw8<TI> raw = next;
    if (it + SLOTS < items) next = source(it + SLOTS);
    const int row = it / H, h = it - row * H;
    const int64_t t = row0 + row;
    const bool key = h >= a.Hq;
    int64_t place = 0;
    if (CACHE && key) {
      place = rows_at[row];
      if (place < 0) continue;  // (a head's lanes together)
      place += (int64_t)(h - a.Hq - (h >= a.Hq + a.Hk ? a.Hk : 0)) * a.page;
      if (h >= a.Hq + a.Hk) {
        if (me.live) straw8<TI>((TI*)a.vp + place * a.D + me.c, raw);
        continue;
      }
    }
    const F8 v = cvt8<TI>(raw);
    float ss = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) ss = fmaf(v.v[j], v.v[j], ss);
    ss = head_sum<LH>(me.live ? ss : 0.f);
    const float rs = 1.f / sqrtf(ss / (float)a.D + a.eps);
    F8 o;
#pragma unroll
    for (int j = 0; j < 8; ++j) o.v[j] = v.v[j] * rs * (key ? wk.v[j] : wq.v[j]);
    if constexpr (ADJ) {
      if (me.turned) {
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
          const float2 g = cs[row * (a.R / 2) + me.ang + j / 2];
          const float x = o.v[j], y = o.v[j + 1];
          o.v[j] = fmaf(x, g.x, -(y * g.y));
          o.v[j + 1] = fmaf(x, g.y, y * g.x);
        }
      }
    } else {
      const F8 u = cvt8<TI>(lane_away<TI>(raw, me.away));
      if (me.turned) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float2 g = cs[row * (a.R / 2) + me.ang + j];
          const float other = u.v[j] * rs * (key ? ok.v[j] : oq.v[j]);
          o.v[j] = fmaf(o.v[j], g.x, me.sign * other * g.y);
        }
      }
    }
    if (me.live) {
      if (CACHE && key) st8<TI>((TI*)a.kp + place * a.D + me.c, o);
      else if (key) st8nt<TI>((TI*)a.ko + t * a.ko_rs + (h - a.Hq) * a.D + me.c, o);
      else st8nt<TI>((TI*)a.qo + t * a.qo_rs + h * a.D + me.c, o);
    }
  }
}

// Workgroups walk over the rows, their share of dwq and dwk in registers; partials [dwq | dwk][workgroup][D].
template <typename TI, int LH, bool ADJ> __global__ __launch_bounds__(RNT) void k_rope_bwd(RopeArgs a, int rb) {
  __shared__ float2 cs[RROWS * 128];
  __shared__ __align__(16) float part[RNT * 8];
  const RopePlace me(LH, a.D, a.R, ADJ);
  const int H = a.Hq + a.Hk;
  constexpr int SLOTS = RNT / LH;
  const F8 wq = rope_weight(a.wq, me.c, me.live), wk = rope_weight(a.wk, me.c, me.live);
  F8 dq = zero8(), dk = zero8();
  for (int64_t row0 = (int64_t)blockIdx.x * rb; row0 < a.rows; row0 += (int64_t)gridDim.x * rb) {
    const int nrows = (int)(a.rows - row0 < rb ? a.rows - row0 : rb), items = nrows * H;
    auto source = [&](int it, bool grad) {
      const int row = it / H, h = it - row * H;
      const int64_t t = row0 + row;
      const TI* p = h < a.Hq ? (grad ? (const TI*)a.gq + t * a.gq_rs : (const TI*)a.q + t * a.q_rs) + h * a.D
                             : (grad ? (const TI*)a.gk + t * a.gk_rs : (const TI*)a.k + t * a.k_rs) + (h - a.Hq) * a.D;
      return ldraw8<true, TI>(p + (me.live ? me.c : 0));
    };
    int it = (int)threadIdx.x / LH;
    Raw8<TI> nv, ng;
    if (it < items) {
      nv = source(it, false);
      ng = source(it, true);
    }
    __syncthreads();  // the rows before are done with their angles
    rope_angles(a, row0, nrows, cs);
    __syncthreads();
    for (; it < items; it += SLOTS) {
      const Raw8<TI> rv = nv, rg = ng;
      if (it + SLOTS < items) {
        nv = source(it + SLOTS, false);
        ng = source(it + SLOTS, true);
      }
      const int row = it / H, h = it - row * H;
      const int64_t t = row0 + row;
      const bool key = h >= a.Hq;
      const F8 v = cvt8<TI>(rv);
      F8 g = cvt8<TI>(rg);
      if constexpr (ADJ) {
        if (me.turned) {
#pragma unroll
          for (int j = 0; j < 8; j += 2) {
            const float2 q = cs[row * (a.R / 2) + me.ang + j / 2];
            const float x = g.v[j], y = g.v[j + 1];
            g.v[j] = x * q.x + y * q.y;
            g.v[j + 1] = y * q.x - x * q.y;
          }
        }
      } else {
        const F8 u = cvt8<TI>(lane_away<TI>(rg, me.away));
        if (me.turned) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float2 q = cs[row * (a.R / 2) + me.ang + j];
            g.v[j] = g.v[j] * q.x - me.sign * u.v[j] * q.y;
          }
        }
      }
      float ss = 0.f, tv = 0.f;
      F8 tw;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        tw.v[j] = g.v[j] * (key ? wk.v[j] : wq.v[j]);
        ss += v.v[j] * v.v[j];
        tv += tw.v[j] * v.v[j];
      }
      ss = head_sum<LH>(me.live ? ss : 0.f);
      tv = head_sum<LH>(me.live ? tv : 0.f);
      const float rs = 1.f / sqrtf(ss / (float)a.D + a.eps), m = tv * rs / (float)a.D;
      F8 o;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float n = v.v[j] * rs, d = g.v[j] * n;
        o.v[j] = rs * (tw.v[j] - n * m);
        dq.v[j] += key ? 0.f : d;
        dk.v[j] += key ? d : 0.f;
      }
      if (me.live) {
        if (key) st8nt<TI>((TI*)a.ko + t * a.ko_rs + (h - a.Hq) * a.D + me.c, o);
        else st8nt<TI>((TI*)a.qo + t * a.qo_rs + h * a.D + me.c, o);
      }
    }
  }
  if (!a.ws) return;
  for (int which = 0; which < 2; ++which) {
    __syncthreads();
    st8<float>(part + (int)threadIdx.x * 8, which ? dk : dq);
    __syncthreads();
    for (int c = (int)threadIdx.x; c < a.D; c += RNT) {
      float s = 0.f;
      for (int k = 0; k < SLOTS; ++k) s += part[k * LH * 8 + c];
      a.ws[((int64_t)which * gridDim.x + blockIdx.x) * a.D + c] = s;
    }
  }
}

// ------------------------------------------------------------------ launches
// Rows of a workgroup: two keep more loads in flight (16384 rows of 28 heads of 256: forward 87 us, backward 126; with one 90
// and 135, with four 92 and 131), one spreads small batches (a training step's kernels, 28 heads of 256: 300 rows 20 us with one, 23 with
// two; 1001 rows 26 and 28; 2047 39 and 36; 3000 51 and 52).
static int rope_rows(const RopeArgs& a) { return a.rows >= 2048 ? RROWS : 1; }
static int rope_bwd_grid(const RopeArgs& a) {
  const int64_t blocks = (a.rows + rope_rows(a) - 1) / rope_rows(a);
  return (int)(blocks < 2048 ? (blocks < 1 ? 1 : blocks) : 2048);
}
size_t rope_bwd_ws_bytes(const RopeArgs& a) { return (size_t)rope_bwd_grid(a) * 2 * a.D * sizeof(float); }

template <typename TI, int LH, bool ADJ> static hipError_t rope_go(RopeKind kind, const RopeArgs& a, hipStream_t s) {
  const int rb = rope_rows(a);
  if (kind == ROPE_BWD) {
    const int grid = rope_bwd_grid(a);
    traced("k_rope_bwd", s, [&] { k_rope_bwd<TI, LH, ADJ><<<grid, RNT, 0, s>>>(a, rb); });
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || !a.ws) return e;
    return launch_colsum(a.ws, grid, a.D, ColsumOut{{a.dwq, a.dwk, nullptr}}, 2, s);
  }
  if (a.rows == 0) return hipSuccess;
  const unsigned grid = (unsigned)((a.rows + rb - 1) / rb);
  traced(kind == ROPE_FWD ? "k_rope_fwd" : "k_rope_cache", s, [&] {
    if (kind == ROPE_FWD) k_rope_fwd<TI, LH, ADJ, false><<<grid, RNT, 0, s>>>(a, rb);
    else k_rope_fwd<TI, LH, ADJ, true><<<grid, RNT, 0, s>>>(a, rb);
  });
  return hipGetLastError();
}
template <typename TI, int LH> static hipError_t rope_adj(RopeKind kind, const RopeArgs& a, hipStream_t s) {
  return a.adjacent ? rope_go<TI, LH, true>(kind, a, s) : rope_go<TI, LH, false>(kind, a, s);
}
template <typename TI> static hipError_t rope_lh(RopeKind kind, const RopeArgs& a, hipStream_t s) {
  if (a.D <= 32) return rope_adj<TI, 4>(kind, a, s);
  if (a.D <= 64) return rope_adj<TI, 8>(kind, a, s);
  if (a.D <= 128) return rope_adj<TI, 16>(kind, a, s);
  return rope_adj<TI, 32>(kind, a, s);
}
hipError_t launch_rope(RopeKind kind, const RopeArgs& a, int dtype, hipStream_t s) {
  return dtype == 0 ? rope_lh<float>(kind, a, s) : rope_lh<__bf16>(kind, a, s);
}

}  // namespace gdn
