// ssm_grad.hip -- gradients of the selective state space scan inside each chunk, on gfx950.
//
// One workgroup per (chunk, group of heads that share b and c), walking over the group's heads.
// With Q = dy x^T, W = Gamma o G o Q (no step), E = S dy and F = dS x (S the state at the chunk's
// start, dS the adjoint at its end, both float32), e_j = 2^(gamma_n - gamma_j):
//   dc_i = sum_h [ sum_j Gamma_ij D_j Q_ij b_j + 2^gamma_i E_i ]
//   db_j = sum_h [ sum_i Gamma_ij D_j Q_ij c_i + e_j D_j F_j ]
//   q_t = d loss / d log a_t = sum_{i >= t} (row_i - D_i col_i + 2^gamma_i c_i . E_i)
//                              + sum_{j < t} D_j e_j b_j . F_j + 2^gamma_n <S, dS>
//   dD_j = W_jj + col_j + e_j b_j . F_j - exp(a_log) q_j,   ddt = dD sigmoid(dt + dt_bias)
// with row_i = sum_{j < i} D_j W_ij and col_j = sum_{i > j} W_ij: what row_i and D_j col_j add for pairs
// on one side of t cancels, and the diagonal, which alone carries no decay, is left out of both (under
// strong decays it would drown q). The two products with Gamma D Q are linear in
// it, so they run once per group on the sum over its heads. b, c, x, dy are exact as bfloat16
// operands; the states are split over three (24 bits), so that the float32 results keep float32
// accuracy. Bound by HBM: the two states of a chunk and head are 8 Dk Dv bytes.
#include "ssm_common.h"

namespace gdn {

struct GradArgs {
  SsmArgs p;
  const float *sv, *ds;  // [slot][Hv][Dk][Dv]: states at the chunks' starts, adjoints at their ends
  float* part;           // [3][slots][Hv]: da_log, ddt_bias, dd_skip of each chunk
  int nslab;
  int64_t slots;
};

template <typename TI, int DK>
__global__ __launch_bounds__(256, 2) void k_ssm_grad(GradArgs a) {
  const SsmArgs& p = a.p;
  constexpr int NDT = DK / 16, KSD = ks_of<TI, DK>(), NSD = DK / KSD, KSC = ks_of<TI, SC>(), NSC = SC / KSC;
  constexpr int NS = ssm_split<TI>(), KE = Mf<TI, KSC>::KE;
  // tiles of a [Dk][64 tokens] product: DT tiles along Dk, TT along the tokens for each wave
  constexpr int DT = NDT >= 4 ? NDT / 4 : 1, TT = NDT >= 4 ? 4 : NDT;
  using LK = Swz<TI, DK, true>;
  using LX = Swz<TI, SP, true>;
  __shared__ __align__(16) TI sB[SC * DK];
  __shared__ __align__(16) TI sC[SC * DK];
  __shared__ __align__(16) TI sX[SC * SP];
  __shared__ __align__(16) TI sY[SC * SP];
  __shared__ __align__(16) TI sR[SC * SC];
  __shared__ __align__(16) float sh[2][6][SC];  // gamma, its remainder, step, 2^gamma, e, dt + bias
  __shared__ float sbn[2];
  __shared__ float srow[10][16], scol[10][16], sdiag[SC], sE[4][SC], sF[4][SC], sfr[4], sdd[4];

  const int kh = (int)(blockIdx.x % p.Hk);
  const int64_t slot = blockIdx.x / p.Hk;
  const int w = wave_id(), l = lane_id(), g = l >> 4, r = l & 15;
  // the slot's sequence: the largest n whose first slot is not behind it
  int n = 0;
  int64_t lo, hi;
  for (int top = p.N; top - n > 1;) {
    const int m = (n + top) >> 1;
    ssm_seq(p.cu, p.T, p.T_total, m, lo, hi);
    if (lo / SC + m <= slot) n = m; else top = m;
  }
  ssm_seq(p.cu, p.T, p.T_total, n, lo, hi);
  const int64_t k = slot - (lo / SC + n);
  if (k < 0 || k >= (hi - lo + SC - 1) / SC) {  // a slot of no chunk
    for (int i = threadIdx.x; i < 3 * p.r; i += 256)
      a.part[((int64_t)(i / p.r) * a.slots + slot) * p.Hv + kh * p.r + i % p.r] = 0.f;
    return;
  }
  const int64_t t0 = lo + k * SC;
  const int len = (int)(hi - t0 < SC ? hi - t0 : SC);

  {
    TileRegs<TI, DK, LK, 256> rb, rc;
    rb.init(p.b_rs, DK);
    rc.init(p.c_rs, DK);
    rb.template load<false>((const TI*)p.b + t0 * p.b_rs + kh * DK, len);
    rc.template load<false>((const TI*)p.c + t0 * p.c_rs + kh * DK, len);
    for (int i = threadIdx.x; i < SC * SC; i += 256) sR[i] = (TI)0.f;
    for (int i = threadIdx.x; i < 4 * SC; i += 256) sE[i / SC][i % SC] = sF[i / SC][i % SC] = 0.f;
    rb.store(sB);
    rc.store(sC);
  }
  lds_barrier();
  // this wave's tiles of the lower triangle: token tiles it >= jt; element e of a lane is (i, j) =
  // (16 it + r, 16 jt + 4 g + e)
  int it[3], jt[3];
  f32x4 G[3], R[3];
#pragma unroll
  for (int u = 0; u < 3; ++u) {
    const int idx = w + 4 * u;
    it[u] = idx >= 6 ? 3 : idx >= 3 ? 2 : idx >= 1 ? 1 : 0;
    jt[u] = idx - it[u] * (it[u] + 1) / 2;
    G[u] = R[u] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (idx >= 10) continue;
#pragma unroll
    for (int s = 0; s < NSD; ++s)
      G[u] = Mf<TI, KSD>::run(ld_n<TI, KSD, STD, LK>(sB, 16 * jt[u], s), ld_n<TI, KSD, STD, LK>(sC, 16 * it[u], s), G[u]);
  }
  auto dtile = [&](int x) { return NDT >= 4 ? w * DT + x : w % NDT; };
  auto ttile = [&](int y) { return NDT >= 4 ? y : (w / NDT) * TT + y; };
  f32x4 dC[DT][TT], dB[DT][TT];
  zero(dC);
  zero(dB);

  for (int hh = 0; hh < p.r; ++hh) {
    const int h = kh * p.r + hh, buf = hh & 1;
    f32x4 E[DT][TT], F[DT][TT], Q[3];
    zero(E);
    zero(F);
#pragma unroll
    for (int u = 0; u < 3; ++u) Q[u] = f32x4{0.f, 0.f, 0.f, 0.f};
    float frob = 0.f;
    const int64_t base = (slot * p.Hv + h) * (int64_t)DK * p.Dv;
    for (int slab = 0; slab < a.nslab; ++slab) {
      const int ncols = p.Dv - slab * SP < SP ? p.Dv - slab * SP : SP;
      {
        TileRegs<TI, SP, LX, 256> rx, ry;
        rx.init(p.x_rs, ncols);
        ry.init(p.dy_rs, ncols);
        rx.template load<true>((const TI*)p.x + t0 * p.x_rs + (int64_t)h * p.Dv + slab * SP, len);
        ry.template load<true>((const TI*)p.dy + t0 * p.dy_rs + (int64_t)h * p.Dv + slab * SP, len);
        lds_barrier();  // the previous rows are used up
        rx.store(sX);
        ry.store(sY);
      }
      if (w == 3 && slab == 0) {
        const float dt = l < len ? p.dt[(t0 + l) * p.Hv + h] : 0.f;
        const Gate q = chunk_gate(dt, p.dt_bias ? p.dt_bias[h] : 0.f, -expf(p.a_log[h]) * kLog2e, l < len);
        const float h32 = (float)q.gam;
        sh[buf][0][l] = h32;
        sh[buf][1][l] = (float)(q.gam - (double)h32);
        sh[buf][2][l] = q.step;
        sh[buf][3][l] = __builtin_amdgcn_exp2f(h32);
        sh[buf][4][l] = __builtin_amdgcn_exp2f((float)(q.tot - q.gam));
        sh[buf][5][l] = q.z;
        if (l == 63) sbn[buf] = __builtin_amdgcn_exp2f((float)q.tot);
      }
      lds_barrier();
#pragma unroll
      for (int x = 0; x < DT; ++x) {
        // rows d = 16 dtile + r of both states, eight (or one) adjacent columns per step
        const int64_t off = base + (int64_t)(16 * dtile(x) + r) * p.Dv + slab * SP;
#pragma unroll
        for (int s = 0; s < NSC; ++s) {
          const int c = kidx<KSC, STD>(s, g, 0);
          float vs[KE], vd[KE];
#pragma unroll
          for (int j = 0; j < KE; ++j) vs[j] = vd[j] = 0.f;
          if (c < ncols) {
            if constexpr (KE == 1) {
              vs[0] = a.sv[off + c];
              vd[0] = a.ds[off + c];
            } else {
#pragma unroll
              for (int j = 0; j < KE; j += 4) {
                const f32x4 p4 = __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(a.sv + off + c + j));
                const f32x4 q4 = __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(a.ds + off + c + j));
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  vs[j + e] = p4[e];
                  vd[j + e] = q4[e];
                }
              }
            }
          }
          if (NDT >= 4 || w < NDT) {
#pragma unroll
            for (int j = 0; j < KE; ++j) frob += vs[j] * vd[j];
          }
          FragT<TI, KSC> fs[NS], fd[NS];
          split_frag<TI, KSC, NS>(vs, fs);
          split_frag<TI, KSC, NS>(vd, fd);
#pragma unroll
          for (int y = 0; y < TT; ++y) {
            const FragT<TI, KSC> yf = ld_n<TI, KSC, STD, LX>(sY, 16 * ttile(y), s);
            const FragT<TI, KSC> xf = ld_n<TI, KSC, STD, LX>(sX, 16 * ttile(y), s);
#pragma unroll
            for (int m = NS - 1; m >= 0; --m) {
              E[x][y] = Mf<TI, KSC>::run(fs[m], yf, E[x][y]);
              F[x][y] = Mf<TI, KSC>::run(fd[m], xf, F[x][y]);
            }
          }
        }
      }
#pragma unroll
      for (int u = 0; u < 3; ++u) {
        if (w + 4 * u >= 10) continue;
#pragma unroll
        for (int s = 0; s < NSC; ++s)
          Q[u] = Mf<TI, KSC>::run(ld_n<TI, KSC, STD, LX>(sX, 16 * jt[u], s), ld_n<TI, KSC, STD, LX>(sY, 16 * it[u], s), Q[u]);
      }
    }
    const float(*gt)[SC] = sh[buf];
    float dd = 0.f;
#pragma unroll
    for (int u = 0; u < 3; ++u) {
      if (w + 4 * u >= 10) continue;
      const int i = 16 * it[u] + r, j0 = 16 * jt[u] + 4 * g;
      const float ih = gt[0][i], il = gt[1][i];
      const f32x4 jh = ld4(&gt[0][j0]), jl = ld4(&gt[1][j0]), st = ld4(&gt[2][j0]);
      float row = 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float gm = i >= j0 + e ? __builtin_amdgcn_exp2f((ih - jh[e]) + (il - jl[e])) : 0.f;
        const float gq = i >= j0 + e ? gm * Q[u][e] : 0.f;
        R[u][e] += gq * st[e];
        float wv = gq * G[u][e];
        if (i == j0 + e) {
          dd += Q[u][e];
          sdiag[i] = wv;
          wv = 0.f;
        }
        row += wv * st[e];
        const float cs = row16_sum(wv);
        if (r == 0) scol[w + 4 * u][4 * g + e] = cs;
      }
      row += __shfl_xor(row, 16);
      row += __shfl_xor(row, 32);
      if (g == 0) srow[w + 4 * u][r] = row;
    }
#pragma unroll
    for (int y = 0; y < TT; ++y) {
      const int t = 16 * ttile(y) + r;
      const float eb = gt[3][t], ed = gt[4][t] * gt[2][t];
      float ce = 0.f, bf = 0.f;
#pragma unroll
      for (int x = 0; x < DT; ++x) {
        const int d0 = 16 * dtile(x) + 4 * g;
        const f32x4 cv = ld4<TI>(sC + LK::at(t, d0)), bv = ld4<TI>(sB + LK::at(t, d0));
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          ce += cv[e] * E[x][y][e];
          bf += bv[e] * F[x][y][e];
        }
        dC[x][y] += eb * E[x][y];
        dB[x][y] += ed * F[x][y];
      }
      ce += __shfl_xor(ce, 16);
      ce += __shfl_xor(ce, 32);
      bf += __shfl_xor(bf, 16);
      bf += __shfl_xor(bf, 32);
      if (g == 0) {
        sE[w][t] = ce;
        sF[w][t] = bf;
      }
    }
    frob = wave_sum(frob);
    dd = wave_sum(dd);
    if (l == 0) {
      sfr[w] = frob;
      sdd[w] = dd;
    }
    lds_barrier();
    if (w == 0) {  // one token per lane
      const int ti = l >> 4;
      float row = 0.f, col = 0.f;
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        if (x <= ti) row += srow[ti * (ti + 1) / 2 + x][r];
        if (x >= ti) col += scol[x * (x + 1) / 2 + ti][r];
      }
      const float step = gt[2][l], z = gt[5][l];
      const float ce = gt[3][l] * (sE[0][l] + sE[1][l] + sE[2][l] + sE[3][l]);
      const float bf = gt[4][l] * (sF[0][l] + sF[1][l] + sF[2][l] + sF[3][l]);
      const float before = __shfl_up(wave_scan_incl(step * bf), 1);  // (the last token's own term carries no decay)
      const float q = wave_rscan_incl(row - step * col + ce) + (l > 0 ? before : 0.f) +
                      sbn[buf] * (sfr[0] + sfr[1] + sfr[2] + sfr[3]);
      const float na = -expf(p.a_log[h]);
      const bool live = l < len;
      const float ddt = live ? (sdiag[l] + col + bf + na * q) / (1.f + expf(-z)) : 0.f;
      if (live) p.ddt[(t0 + l) * p.Hv + h] = ddt;
      const float da = wave_sum(live ? q * step * na : 0.f), db = wave_sum(ddt);
      if (l == 0) {
        const int64_t at = slot * p.Hv + h, plane = a.slots * p.Hv;
        a.part[at] = da;
        a.part[plane + at] = db;
        a.part[2 * plane + at] = sdd[0] + sdd[1] + sdd[2] + sdd[3];
      }
    }
  }
  // the heads' sum of Gamma D Q, and its products with b and c
#pragma unroll
  for (int u = 0; u < 3; ++u)
    if (w + 4 * u < 10) st4<TI>(sR + LX::at(16 * it[u] + r, 16 * jt[u] + 4 * g), R[u]);
  lds_barrier();
#pragma unroll
  for (int s = 0; s < NSC; ++s) {
    FragT<TI, KSC> bf[DT], cf[DT];
#pragma unroll
    for (int x = 0; x < DT; ++x) {
      bf[x] = ld_t<TI, KSC, STD, LK>(sB, 16 * dtile(x), s);
      cf[x] = ld_t<TI, KSC, STD, LK>(sC, 16 * dtile(x), s);
    }
#pragma unroll
    for (int y = 0; y < TT; ++y) {
      const FragT<TI, KSC> rn = ld_n<TI, KSC, STD, LX>(sR, 16 * ttile(y), s);
      const FragT<TI, KSC> rt = ld_t<TI, KSC, STD, LX>(sR, 16 * ttile(y), s);
#pragma unroll
      for (int x = 0; x < DT; ++x) {
        dC[x][y] = Mf<TI, KSC>::run(bf[x], rn, dC[x][y]);
        dB[x][y] = Mf<TI, KSC>::run(cf[x], rt, dB[x][y]);
      }
    }
  }
#pragma unroll
  for (int y = 0; y < TT; ++y) {
    const int t = 16 * ttile(y) + r;
    if (t >= len) continue;
#pragma unroll
    for (int x = 0; x < DT; ++x) {
      const int d0 = kh * DK + 16 * dtile(x) + 4 * g;
      st4<TI>((TI*)p.dc + (t0 + t) * p.dc_rs + d0, dC[x][y]);
      st4<TI>((TI*)p.db + (t0 + t) * p.db_rs + d0, dB[x][y]);
    }
  }
}

template <typename TI> static hipError_t grad_d(const GradArgs& a, hipStream_t s) {
  const unsigned grid = (unsigned)(a.slots * a.p.Hk);
  switch (a.p.Dk) {
    case 16: traced("k_ssm_grad", s, [&] { k_ssm_grad<TI, 16><<<grid, 256, 0, s>>>(a); }); break;
    case 32: traced("k_ssm_grad", s, [&] { k_ssm_grad<TI, 32><<<grid, 256, 0, s>>>(a); }); break;
    case 64: traced("k_ssm_grad", s, [&] { k_ssm_grad<TI, 64><<<grid, 256, 0, s>>>(a); }); break;
    case 128: traced("k_ssm_grad", s, [&] { k_ssm_grad<TI, 128><<<grid, 256, 0, s>>>(a); }); break;
    default: return hipErrorInvalidValue;
  }
  return hipGetLastError();
}

hipError_t launch_ssm_grad(const SsmArgs& p, int dtype, const float* ds, float* part, hipStream_t s) {
  GradArgs a;
  a.p = p;
  a.sv = p.sv;
  a.ds = ds;
  a.part = part;
  a.nslab = (p.Dv + SP - 1) / SP;
  a.slots = ssm_slots(p.T_total, p.N);
  return dtype == 0 ? grad_d<float>(a, s) : grad_d<__bf16>(a, s);
}

}  // namespace gdn
