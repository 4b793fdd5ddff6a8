// norm.hip -- RMS norms around a block, fused with the gate behind it and with the residual
// addition before the next one, forward and backward, on gfx950.
//
// Per group of W values, with r = 1 / sqrt(mean(v^2) + eps) and n = v r:
//   gated:       y = n w silu(z) of v = x,  or  y = n w of v = x silu(z) (gate first)
//   add:         v = res = h + scale s y (as stored),  out = n w
//   backward:    for t = (gradient of n w) w:  dv = r (t - n mean(t n)),  dw = sum_rows (.) n
//                gated: the gate's factor and its derivative silu'(z) = sigma (1 + z (1 - sigma))
//                on either side; add: dh = dv + dres, dy = scale s dh, ds = scale sum_rows dh y
//
// Streaming work: every row element is read and written once, bound by HBM. A group is held in
// registers by NL lanes (eight adjacent values per lane and vector, V vectors): the 64 / L groups
// side by side in one wave up to 2048 values, a whole workgroup beyond. All arithmetic is
// float32; results are rounded once. Measured (bf16, 16384 rows): gated norm of 48 x 128 forward 126 us
// (4.8 TB/s), backward 215 + 6 us (4.7); add norm of 5120 forward 130 us (5.2), backward 203 + 9 us (5.0). float32, 8192
// rows: gated norm 118 and 224 + 6 us, add norm 140 and 236 + 9 us. Lanes to a group are a power of two with 1, 2
// or 4 vectors each, so that widths between waste some (520 values, 65 vectors, take 64 lanes twice).
#include "vec8.h"

namespace gdn {

// Lanes and vectors of a launch. BLK = false: L (a power of two up to 64) lanes per group inside a
// wave of a 256-thread workgroup; BLK = true: the workgroup's NT threads hold one group.
struct NormPlan {
  int L, V, NT;
  bool blk;
};

static NormPlan norm_plan(int W) {
  const int vecs = W / 8;
  NormPlan p;
  if (vecs <= 256) {  // one wave: V = 1, 2 or 4
    p.blk = false;
    p.NT = 256;
    p.L = 1;
    while (p.L < 64 && p.L < vecs) p.L *= 2;
    p.V = vecs <= 64 ? 1 : vecs <= 128 ? 2 : 4;
  } else {
    p.blk = true;
    p.NT = vecs <= 768 ? 256 : 512;
    p.L = p.NT;
    const int v = (vecs + p.NT - 1) / p.NT;
    p.V = v <= 2 ? 2 : v <= 3 ? 3 : 4;
  }
  return p;
}

// Sum over a group's lanes, in every lane (fixed order). `red`: two rows of NT / 64 floats, used
// in turn, so that one barrier per sum is enough.
template <bool BLK, int NT> __device__ __forceinline__ float group_sum(float x, int L, float* red, int& turn) {
  if constexpr (!BLK) {
    for (int o = 1; o < L; o <<= 1) x += __shfl_xor(x, o);
    return x;
  } else {
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) x += __shfl_xor(x, o);
    float* r = red + turn * (NT / 64);
    turn ^= 1;
    if ((threadIdx.x & 63) == 0) r[threadIdx.x >> 6] = x;
    __syncthreads();
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < NT / 64; ++i) s += r[i];
    return s;
  }
}

// The residual before its rounding: product and sum rounded one after the other, as the elementary
// operations are (a fused one would round a few of 10^5 bfloat16 residuals to the other neighbour, which
// every later value then shows).
__device__ __forceinline__ float residual(float h, float f, float y) {
#pragma clang fp contract(off)
  const float p = f * y;
  return h + p;
}

__device__ __forceinline__ float silu_grad(float z, float sg) { return sg * (1.f + z * (1.f - sg)); }

// ------------------------------------------------------------------ forward
// One group per slot (wave lanes or workgroup); slots take the groups of the rows in order (a
// grid of at most kMaxBlocks walks over more).
constexpr int64_t kMaxBlocks = 1 << 20;

template <typename TI, int V, bool BLK, int NT, bool ADD>
__global__ __launch_bounds__(NT) void k_norm_fwd(NormArgs a, int L) {
  __shared__ float red[2 * (NT / 64)];
  int turn = 0;
  const int per = BLK ? 1 : NT / L, slot = BLK ? 0 : (int)threadIdx.x / L, li = BLK ? (int)threadIdx.x : (int)threadIdx.x % L;
  const int64_t items = a.rows * a.groups, blocks = (items + per - 1) / per;
  for (int64_t ib = blockIdx.x; ib < blocks; ib += gridDim.x) {
    const int64_t item = ib * per + slot;
    const bool live = item < items;  // whole groups of lanes: the sums below stay within live lanes
    const uint32_t row = live ? (uint32_t)item / (uint32_t)a.groups : 0, g = live ? (uint32_t)item % (uint32_t)a.groups : 0;
    const int W = a.width, gc = (int)g * W;
    const TI* x = (const TI*)a.x + (int64_t)row * a.x_rs + gc;
    const TI* z = (const TI*)a.z + (int64_t)row * a.z_rs + gc;
    Raw8<TI> rx[V], rz[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int c = (li + j * L) * 8;
      if (live && c < W) {
        rx[j] = ldraw8<true, TI>(x + c);
        rz[j] = ldraw8<true, TI>(z + c);
      }
    }
    F8 v[V], gt[V];
    float ss = 0.f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int c = (li + j * L) * 8;
      v[j] = zero8();
      if (!live || c >= W) continue;
      const F8 xx = cvt8<TI>(rx[j]), zz = cvt8<TI>(rz[j]);
      if constexpr (ADD) {
        F8 sv;
        if (a.s) sv = ld8<float>(a.s + c);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float f = a.s ? a.scale * sv.v[i] : a.scale;
          v[j].v[i] = (float)(TI)residual(xx.v[i], f, zz.v[i]);  // as the residual is stored
        }
        st8<TI>((TI*)a.o + (int64_t)row * a.o_rs + c, v[j]);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          gt[j].v[i] = zz.v[i] * sigmoidf<TI>(zz.v[i]);
          v[j].v[i] = a.gate_first ? xx.v[i] * gt[j].v[i] : xx.v[i];
        }
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) ss += v[j].v[i] * v[j].v[i];
    }
    const float r = 1.f / sqrtf(group_sum<BLK, NT>(ss, L, red, turn) / (float)W + a.eps);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int c = (li + j * L) * 8;
      if (!live || c >= W) continue;
      const F8 w = ld8<float>(a.w + (a.shared ? c : gc + c));
      F8 o;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        o.v[i] = v[j].v[i] * r * w.v[i];
        if constexpr (!ADD)
          if (!a.gate_first) o.v[i] *= gt[j].v[i];
      }
      if constexpr (ADD)
        st8<TI>((TI*)a.o2 + (int64_t)row * a.o2_rs + c, o);
      else
        st8<TI>((TI*)a.o + (int64_t)row * a.o_rs + gc + c, o);
    }
  }
}

// ------------------------------------------------------------------ backward
// A workgroup keeps `gpb` groups and walks down the rows, rpp at a time (slot = row in the pass,
// group), its share of dw (and ds) in registers; at the end the rows' shares are added in LDS and
// written as one partial per workgroup, summed by k_colsum: no atomics, a fixed order.
// Grid (group blocks, row splits). Partials: shared weights [splits * blocks][W], else
// [splits][groups W]; ds behind them in the same form.
template <typename TI, int V, bool BLK, int NT, bool ADD>
__global__ __launch_bounds__(NT) void k_norm_bwd(NormArgs a, int L, int gpb) {
  __shared__ float red[2 * (NT / 64)];
  __shared__ __align__(16) float part[BLK ? 4 : NT * V * 8];
  int turn = 0;
  const int slots = BLK ? 1 : NT / L, slot = BLK ? 0 : (int)threadIdx.x / L;
  const int li = BLK ? (int)threadIdx.x : (int)threadIdx.x % L;
  const int rpp = slots / gpb, rs = slot / gpb, g = (int)blockIdx.x * gpb + slot % gpb;
  const int W = a.width, gc = g * W;
  const bool mine = rs < rpp && g < a.groups;
  F8 w[V], sv[V], dw[V], ds[V];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int c = (li + j * L) * 8;
    dw[j] = ds[j] = zero8();
    if (mine && c < W) {
      w[j] = ld8<float>(a.w + (a.shared ? c : gc + c));
      if constexpr (ADD) {
#pragma unroll
        for (int i = 0; i < 8; ++i) sv[j].v[i] = a.scale * (a.s ? a.s[c + i] : 1.f);
      }
    }
  }
  const int64_t step = (int64_t)gridDim.y * rpp;
  // every thread takes the same number of turns (the sums of a workgroup-wide group hold barriers)
  for (int64_t row0 = (int64_t)blockIdx.y * rpp; row0 < a.rows; row0 += step) {
    const int64_t row = row0 + rs;
    const bool live = mine && row < a.rows;
    const TI* x = (const TI*)a.x + row * a.x_rs + gc;
    const TI* z = (const TI*)a.z + row * a.z_rs + gc;
    const TI* gy = (const TI*)a.g + row * a.g_rs + gc;
    const TI* g2 = (const TI*)a.g2 + row * a.g2_rs + gc;
    Raw8<TI> rx[V], rz[V], rg[V], r2[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int c = (li + j * L) * 8;
      if (live && c < W) {
        rx[j] = ldraw8<true, TI>(x + c);
        rg[j] = ldraw8<true, TI>(gy + c);
        if (!ADD || a.ds) rz[j] = ldraw8<true, TI>(z + c);
        if (ADD && a.g2) r2[j] = ldraw8<true, TI>(g2 + c);
      }
    }
    F8 v[V], dy[V], sg[V];
    float ss = 0.f, tv = 0.f;  // sum v^2 and sum t v
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int c = (li + j * L) * 8;
      v[j] = dy[j] = zero8();
      if (!live || c >= W) continue;
      v[j] = cvt8<TI>(rx[j]);
      dy[j] = cvt8<TI>(rg[j]);
      if constexpr (!ADD) {
        const F8 zz = cvt8<TI>(rz[j]);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          sg[j].v[i] = sigmoidf<TI>(zz.v[i]);
          const float gt = zz.v[i] * sg[j].v[i];
          if (a.gate_first) v[j].v[i] *= gt;
          const float dn = a.gate_first ? dy[j].v[i] : dy[j].v[i] * gt;
          ss += v[j].v[i] * v[j].v[i];
          tv += dn * w[j].v[i] * v[j].v[i];
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          ss += v[j].v[i] * v[j].v[i];
          tv += dy[j].v[i] * w[j].v[i] * v[j].v[i];
        }
      }
    }
    ss = group_sum<BLK, NT>(ss, L, red, turn);
    tv = group_sum<BLK, NT>(tv, L, red, turn);
    const float r = 1.f / sqrtf(ss / (float)W + a.eps);
    const float m = tv * r / (float)W;  // mean(t n)
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int c = (li + j * L) * 8;
      if (!live || c >= W) continue;
      F8 o, o2;
      if constexpr (!ADD) {
        const F8 zz = cvt8<TI>(rz[j]), xx = cvt8<TI>(rx[j]);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float n = v[j].v[i] * r, gt = zz.v[i] * sg[j].v[i], gd = silu_grad(zz.v[i], sg[j].v[i]);
          const float dn = a.gate_first ? dy[j].v[i] : dy[j].v[i] * gt;
          const float dv = r * (dn * w[j].v[i] - n * m);
          dw[j].v[i] += dn * n;
          o.v[i] = a.gate_first ? dv * gt : dv;
          o2.v[i] = (a.gate_first ? dv * xx.v[i] : dy[j].v[i] * n * w[j].v[i]) * gd;
        }
        st8nt<TI>((TI*)a.o + row * a.o_rs + gc + c, o);
        st8nt<TI>((TI*)a.o2 + row * a.o2_rs + gc + c, o2);
      } else {
        F8 yy, up = zero8();
        if (a.ds) yy = cvt8<TI>(rz[j]);
        if (a.g2) up = cvt8<TI>(r2[j]);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float n = v[j].v[i] * r;
          o.v[i] = r * (dy[j].v[i] * w[j].v[i] - n * m) + up.v[i];
          dw[j].v[i] += dy[j].v[i] * n;
          if (a.ds) ds[j].v[i] += o.v[i] * yy.v[i];
          o2.v[i] = sv[j].v[i] * o.v[i];
        }
        st8nt<TI>((TI*)a.o + row * a.o_rs + c, o);
        if (a.o2) st8nt<TI>((TI*)a.o2 + row * a.o2_rs + c, o2);
      }
    }
  }
  // the workgroup's partials
  const int64_t wfull = a.shared ? W : (int64_t)a.groups * W;
  const int64_t prow = a.shared ? (int64_t)blockIdx.y * gridDim.x + blockIdx.x : blockIdx.y;
  const int64_t nrow = a.shared ? (int64_t)gridDim.x * gridDim.y : gridDim.y;
  for (int which = 0; which < (ADD ? 2 : 1); ++which) {
    if (which == 0 ? !a.dw : !a.ds) continue;
    float* dst = a.ws + (which == 1 && a.dw ? nrow * wfull : 0) + prow * wfull;
    if constexpr (BLK) {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int c = (li + j * L) * 8;
        if (c < W) {
          F8 q = which ? ds[j] : dw[j];
          if (which)
#pragma unroll
            for (int i = 0; i < 8; ++i) q.v[i] *= a.scale;
          st8<float>(dst + (a.shared ? c : gc + c), q);
        }
      }
    } else {
      __syncthreads();
      const int WP = V * L * 8;  // floats of a slot's share
#pragma unroll
      for (int j = 0; j < V; ++j) st8<float>(part + slot * WP + (li + j * L) * 8, which ? ds[j] : dw[j]);
      __syncthreads();
      const int gl = min(gpb, a.groups - (int)blockIdx.x * gpb);  // groups of this workgroup
      if (a.shared) {
        for (int c = threadIdx.x; c < W; c += NT) {
          float q = 0.f;
          for (int k = 0; k < rpp * gpb; ++k)
            if (k % gpb < gl) q += part[k * WP + c];
          dst[c] = which ? q * a.scale : q;
        }
      } else {
        for (int c = threadIdx.x; c < gl * W; c += NT) {
          const int gg = c / W, cc = c - gg * W;
          float q = 0.f;
          for (int k = 0; k < rpp; ++k) q += part[(k * gpb + gg) * WP + cc];
          dst[(int64_t)blockIdx.x * gpb * W + c] = which ? q * a.scale : q;
        }
      }
    }
  }
}

// Column sums of the planes [R][W] behind one another (grid y: the plane; its output may be
// nullptr): a workgroup takes 16 columns, 64 threads each walk down every 64th row (a few hundred rows
// of dependent loads are a matter of latency: 16 threads took 9.8 us for 2048 x 128, 64 take 6). Sums
// over tokens cancel: the partials are float32, their sum runs in 64 bits.
__global__ __launch_bounds__(1024) void k_colsum(const float* in, int64_t R, int W, ColsumOut o) {
  __shared__ double part[64][17];
  const int c = (int)(threadIdx.x & 15), k = (int)(threadIdx.x >> 4), col = (int)blockIdx.x * 16 + c;
  float* out = o.p[blockIdx.y];
  if (!out) return;
  in += (int64_t)blockIdx.y * R * W;
  double q = 0.0;
  if (col < W) {
#pragma unroll 8
    for (int64_t r = k; r < R; r += 64) q += (double)in[r * W + col];
  }
  part[k][c] = q;
  __syncthreads();
  if (k < 4) {  // one wave: 16 rows each, then the four of them
    double s = 0.0;
#pragma unroll
    for (int i = 0; i < 16; ++i) s += part[k * 16 + i][c];
    s += __shfl_xor(s, 16);
    s += __shfl_xor(s, 32);
    if (k == 0 && col < W) out[col] = (float)s;
  }
}

hipError_t launch_colsum(const float* in, int64_t R, int W, const ColsumOut& o, int planes, hipStream_t s) {
  traced("k_colsum", s, [&] { k_colsum<<<dim3((unsigned)((W + 15) / 16), (unsigned)planes), 1024, 0, s>>>(in, R, W, o); });
  return hipGetLastError();
}

// ------------------------------------------------------------------ launches
// Backward grid. A workgroup-wide group holds some 200 registers a thread and two rows in flight per
// compute unit's SIMD fill it (two workgroups each; more only cost partials: 16384 x 5120 takes 213 us,
// with four 230); groups inside a wave are small, and eight workgroups keep enough loads in flight
// (16384 x 48 x 128: 216 us, with two 273). No more row splits than passes.
struct BwdGrid {
  int gpb, splits, blocks;
};
static BwdGrid bwd_grid(const NormArgs& a, const NormPlan& p) {
  const int slots = p.blk ? 1 : p.NT / p.L;
  BwdGrid g;
  g.gpb = a.groups < slots ? a.groups : slots;
  g.blocks = (a.groups + g.gpb - 1) / g.gpb;
  const int64_t passes = (a.rows + slots / g.gpb - 1) / (slots / g.gpb);
  int64_t want = ((p.blk ? 512 : 2048) + g.blocks - 1) / g.blocks;
  if (want > passes) want = passes;
  g.splits = (int)(want < 1 ? 1 : want);
  return g;
}

size_t norm_ws_bytes(const NormArgs& a, bool add) {
  const BwdGrid g = bwd_grid(a, norm_plan(a.width));
  const size_t rows = a.shared ? (size_t)g.splits * g.blocks : (size_t)g.splits;
  const size_t W = a.shared ? (size_t)a.width : (size_t)a.groups * a.width;
  return rows * W * sizeof(float) * (add ? 2 : 1);
}

template <typename TI, int V, bool BLK, int NT, bool ADD>
static hipError_t norm_go(bool backward, const NormArgs& a, const NormPlan& p, hipStream_t s) {
  if (!backward) {
    const int per = BLK ? 1 : NT / p.L;
    int64_t blocks = (a.rows * a.groups + per - 1) / per;
    if (blocks == 0) return hipSuccess;
    if (blocks > kMaxBlocks) blocks = kMaxBlocks;
    traced(ADD ? "k_add_norm_fwd" : "k_gated_norm_fwd", s,
           [&] { k_norm_fwd<TI, V, BLK, NT, ADD><<<(unsigned)blocks, NT, 0, s>>>(a, p.L); });
    return hipGetLastError();
  }
  const BwdGrid g = bwd_grid(a, p);
  const dim3 grid((unsigned)g.blocks, (unsigned)g.splits);
  traced(ADD ? "k_add_norm_bwd" : "k_gated_norm_bwd", s,
         [&] { k_norm_bwd<TI, V, BLK, NT, ADD><<<grid, NT, 0, s>>>(a, p.L, g.gpb); });
  hipError_t e = hipGetLastError();
  const int64_t R = a.shared ? (int64_t)g.splits * g.blocks : g.splits;
  const int W = a.shared ? a.width : a.groups * a.width;
  if (e == hipSuccess && a.dw && a.ds)
    e = launch_colsum(a.ws, R, W, ColsumOut{{a.dw, a.ds, nullptr}}, 2, s);
  else if (e == hipSuccess && (a.dw || a.ds))
    e = launch_colsum(a.ws, R, W, ColsumOut{{a.dw ? a.dw : a.ds, nullptr, nullptr}}, 1, s);
  return e;
}

template <typename TI, bool ADD> static hipError_t norm_v(bool backward, const NormArgs& a, hipStream_t s) {
  const NormPlan p = norm_plan(a.width);
  if (!p.blk) {
    if (p.V == 1) return norm_go<TI, 1, false, 256, ADD>(backward, a, p, s);
    if (p.V == 2) return norm_go<TI, 2, false, 256, ADD>(backward, a, p, s);
    return norm_go<TI, 4, false, 256, ADD>(backward, a, p, s);
  }
  if (p.NT == 256) return p.V == 2 ? norm_go<TI, 2, true, 256, ADD>(backward, a, p, s) : norm_go<TI, 3, true, 256, ADD>(backward, a, p, s);
  if (p.V == 2) return norm_go<TI, 2, true, 512, ADD>(backward, a, p, s);
  if (p.V == 3) return norm_go<TI, 3, true, 512, ADD>(backward, a, p, s);
  return norm_go<TI, 4, true, 512, ADD>(backward, a, p, s);
}

hipError_t launch_norm(NormKind kind, const NormArgs& a, int dtype, hipStream_t s) {
  const bool add = kind == ADD_FWD || kind == ADD_BWD, bwd = kind == GATE_BWD || kind == ADD_BWD;
  if (dtype == 0) return add ? norm_v<float, true>(bwd, a, s) : norm_v<float, false>(bwd, a, s);
  return add ? norm_v<__bf16, true>(bwd, a, s) : norm_v<__bf16, false>(bwd, a, s);
}

}  // namespace gdn
