// ssm_grad.hip -- gradients of the selective state space scan inside each chunk, on gfx950.
//
// One workgroup per (chunk, group of heads that share b and c), walking over the group's heads (a part of
// them where there are few chunks, k_ssm_fold).
// With Q = dy x^T, W = Gamma o G o Q (no step), E = S dy and F = dS x (S the state at the chunk's
// start, dS the adjoint at its end, both float32), e_j = 2^(gamma_n - gamma_j):
//   dc_i = sum_h [ sum_j Gamma_ij D_j Q_ij b_j + 2^gamma_i E_i ]
//   db_j = sum_h [ sum_i Gamma_ij D_j Q_ij c_i + e_j D_j F_j ]
//   q_t = d loss / d log a_t = sum_{i >= t} (row_i - D_i col_i + 2^gamma_i c_i . E_i)
//                              + sum_{j < t} D_j e_j b_j . F_j + 2^gamma_n <S, dS>
//   dD_j = W_jj + col_j + e_j b_j . F_j - exp(a_log) q_j,   ddt = dD sigmoid(dt + dt_bias)
// with row_i = sum_{j < i} D_j W_ij and col_j = sum_{i > j} W_ij (what row_i and D_j col_j add for pairs
// on one side of t cancels; the kernel forms that difference within tiles of 16 tokens only). The diagonal,
// which alone carries no decay, is left out of both: under strong decays it would drown q. The two products with Gamma D Q are linear in
// it, so they run once per group on the sum over its heads. b, c, x, dy are exact as bfloat16
// operands; the states are split over three (24 bits), so that the float32 results keep float32
// accuracy, and Gamma D Q over two, so that db and dc carry no rounding but their own.
//
// Bound by HBM: the two states of a chunk and head are 8 Dk Dv bytes. Measured (bf16, 4 x 4096 tokens, 64 heads
// of 128 x 64 in 8 groups): 422 to 457 us for the 1.5 GB of states and rows, which a copy would take 290 us
// to move; the rest is the start of each workgroup (one to a compute unit), which nothing overlaps.
//
// Eight waves: wave w holds 16 rows of Dk (all tokens; with a smaller state some tokens) and one or two
// tiles of the tokens' triangle. The next head's rows and states are on their way while a head is
// computed (a state's registers are refilled as soon as its fragments are split off). What is left of a
// head after its products is one value per token: its sums over lanes and waves, and the scans that give
// q, are done for HB heads at once, one head to a wave, and so are the gates.
#include "ssm_common.h"

namespace gdn {

struct GradArgs {
  SsmArgs p;
  const float *sv, *ds;  // [slot][Hv][Dk][Dv]: states at the chunks' starts, adjoints at their ends
  float* part;           // [3][slots][Hv]: da_log, ddt_bias, dd_skip of each chunk
  float* fold;           // [2][parts][T_total][Hk Dk]: each part's dc and db, where a group has several
  int nslab, parts, hpp; // workgroups to a group, heads of each
  int64_t slots;
};

// The slot's sequence and its chunk there: the largest n whose first slot is not behind it, 64 probes at
// a time (by whole waves). Returns the chunk's rows, none for a slot of no chunk.
__device__ __forceinline__ int slot_chunk(const SsmArgs& p, int64_t slot, int64_t& t0) {
  int n = 0;
  int64_t lo, hi;
  if (p.cu || p.N > 1) {
    for (int m = p.N; m > 1;) {
      const int stride = (m + 63) / 64, i = lane_id() * stride;
      bool in = false;
      if (i < m) {
        int64_t x = p.cu ? (int64_t)p.cu[n + i] : (int64_t)(n + i) * p.T;
        x = x < 0 ? 0 : (x > p.T_total ? p.T_total : x);
        in = x / SC + n + i <= slot;
      }
      const uint64_t hit = __ballot(in);
      const int at = (hit ? 63 - __builtin_clzll(hit) : 0) * stride;
      n += at;
      m = m - at < stride ? m - at : stride;
    }
  }
  ssm_seq(p.cu, p.T, p.T_total, n, lo, hi);
  const int64_t k = slot - (lo / SC + n);
  t0 = lo + k * SC;
  if (k < 0 || k >= (hi - lo + SC - 1) / SC) return 0;
  return (int)(hi - t0 < SC ? hi - t0 : SC);
}

template <typename TI, int DK>
__global__ __launch_bounds__(512, 2) void k_ssm_grad(GradArgs a) {
  const SsmArgs& p = a.p;
  constexpr int NT = 512, NDT = DK / 16, KSD = ks_of<TI, DK>(), NSD = DK / KSD, KSC = ks_of<TI, SC>(), NSC = SC / KSC;
  constexpr int NS = ssm_split<TI>(), KE = Mf<TI, KSC>::KE;
  constexpr int TT = NDT == 8 ? 4 : NDT == 4 ? 2 : 1;   // token tiles of a wave's [16 of Dk][64 tokens] products
  constexpr int HB = sizeof(TI) == 4 ? 2 : 8;           // heads whose scans are done together
  constexpr int XB = sizeof(TI) == 4 ? 1 : 2;           // buffers of x and dy
  using LK = PadRow<TI, DK>;
  using LX = Swz<TI, SP, true>;
  __shared__ __align__(16) TI sB[LK::size(SC)];
  __shared__ __align__(16) TI sC[LK::size(SC)];
  __shared__ __align__(16) TI sXY[XB][2][SC * SP];
  constexpr int NR = sizeof(TI) == 4 ? 1 : 2;           // terms of Gamma D Q as an operand
  __shared__ __align__(16) TI sR[NR][SC * SC];
  __shared__ __align__(16) float sh[2][HB][6][SC];  // gamma, its remainder, step, 2^gamma, e, dt + bias
  __shared__ float sbn[2][HB];
  __shared__ __align__(16) float srow[HB][10][16], scol[HB][10][16];
  __shared__ float sdiag[HB][SC], sE[HB][8][SC], sF[HB][8][SC], sfr[HB][8], sdd[HB][8];

  const int pt = (int)(blockIdx.x % a.parts), kh = (int)(blockIdx.x / a.parts % p.Hk);
  const int64_t slot = blockIdx.x / a.parts / p.Hk;
  const int hd0 = kh * p.r + pt * a.hpp, nhd = min(a.hpp, p.r - pt * a.hpp);  // this workgroup's heads
  const int w = wave_id(), l = lane_id(), g = l >> 4, r = l & 15;
  int64_t t0;
  const int len = slot_chunk(p, slot, t0);
  if (len == 0) {  // a slot of no chunk
    for (int i = threadIdx.x; i < 3 * nhd; i += NT)
      a.part[((int64_t)(i / nhd) * a.slots + slot) * p.Hv + hd0 + i % nhd] = 0.f;
    return;
  }

  const int dtile = w % NDT, ttile0 = (w / NDT) * TT;       // this wave's tiles of the [Dk][tokens] products
  const bool mine = NDT > 1 || w < 4;                       // (a state of 16 rows leaves four waves without)
  const int pairs = nhd * a.nslab;                          // (head, slab) steps

  // rows and states of step q on their way
  TileRegs<TI, SP, LX, NT> rx, ry;
  float rs[NSC][KE], rd[NSC][KE];  // this lane's row of S and dS: 64 columns, KE per step
  auto load_rows = [&](int q) {
    const int h = hd0 + q / a.nslab, slab = q % a.nslab;
    const int ncols = p.Dv - slab * SP < SP ? p.Dv - slab * SP : SP;
    rx.init(p.x_rs, ncols);
    ry.init(p.dy_rs, ncols);
    rx.template load<true>((const TI*)p.x + t0 * p.x_rs + (int64_t)h * p.Dv + slab * SP, len);
    ry.template load<true>((const TI*)p.dy + t0 * p.dy_rs + (int64_t)h * p.Dv + slab * SP, len);
  };
  auto load_state = [&](int q, int s) {
    const int h = hd0 + q / a.nslab, slab = q % a.nslab;
    const int64_t base = (slot * p.Hv + h) * (int64_t)DK * p.Dv;
    const uint32_t bytes = (uint32_t)(DK * p.Dv) * 4u;
    const __amdgpu_buffer_rsrc_t bs = rows_rsrc(a.sv + base, bytes), bd = rows_rsrc(a.ds + base, bytes);
    const int c = slab * SP + kidx<KSC, STD>(s, g, 0);
    const uint32_t voff = mine && c < p.Dv ? (uint32_t)((16 * dtile + r) * p.Dv + c) * 4u : kNowhere;
    if constexpr (KE == 1) {
      rs[s][0] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(bs, (int)voff, 0, 2));
      rd[s][0] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(bd, (int)voff, 0, 2));
    } else {
#pragma unroll
      for (int j = 0; j < KE; j += 4) {
        const f32x4 vs = __builtin_bit_cast(f32x4, buf_ld16<true>(bs, voff + 4u * j));
        const f32x4 vd = __builtin_bit_cast(f32x4, buf_ld16<true>(bd, voff + 4u * j));
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          rs[s][j + e] = vs[e];
          rd[s][j + e] = vd[e];
        }
      }
    }
  };
  // the gates of head hh + w (one head of a batch to a wave)
  float rdt = 0.f;
  auto load_dt = [&](int hh) {
    rdt = w < HB && hh + w < nhd && l < len ? p.dt[(t0 + l) * p.Hv + hd0 + hh + w] : 0.f;
  };
  auto gates = [&](int hh) {
    if (w >= HB || hh + w >= nhd) return;
    const int h = hd0 + hh + w, b = (hh / HB) & 1;
    const Gate q = chunk_gate(rdt, p.dt_bias ? p.dt_bias[h] : 0.f, neg_a_log2(p.a_log[h]), l < len);
    const float h32 = (float)q.gam;
    float(*gt)[SC] = sh[b][w];
    gt[0][l] = h32;
    gt[1][l] = (float)(q.gam - (double)h32);
    gt[2][l] = q.step;
    gt[3][l] = exp2_d(q.gam);
    gt[4][l] = exp2_d(q.tot - q.gam);
    gt[5][l] = q.z;
    if (l == 63) sbn[b][w] = exp2_d(q.tot);
  };

  {
    TileRegs<TI, DK, LK, NT> rb, rc;
    rb.init(p.b_rs, DK);
    rc.init(p.c_rs, DK);
    rb.template load<false>((const TI*)p.b + t0 * p.b_rs + kh * DK, len);
    rc.template load<false>((const TI*)p.c + t0 * p.c_rs + kh * DK, len);
    load_dt(0);
    load_rows(0);
#pragma unroll
    for (int s = 0; s < NSC; ++s) load_state(0, s);
    for (int i = threadIdx.x; i < NR * SC * SC; i += NT) sR[0][i] = (TI)0.f;
    for (int i = threadIdx.x; i < HB * 8 * SC; i += NT) (&sE[0][0][0])[i] = (&sF[0][0][0])[i] = 0.f;
    rb.store(sB);
    rc.store(sC);
    gates(0);
    load_dt(HB);
    rx.store(sXY[0][0]);
    ry.store(sXY[0][1]);
  }
  lds_barrier();
  // this wave's tiles of the lower triangle: token tiles it >= jt; element e of a lane is (i, j) =
  // (16 it + r, 16 jt + 4 g + e)
  int it[2], jt[2];
  f32x4 G[2], R[2], Q[2];
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int idx = w + 8 * u;
    it[u] = idx >= 6 ? 3 : idx >= 3 ? 2 : idx >= 1 ? 1 : 0;
    jt[u] = idx - it[u] * (it[u] + 1) / 2;
    G[u] = R[u] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (idx >= 10) continue;
#pragma unroll
    for (int s = 0; s < NSD; ++s)
      G[u] = Mf<TI, KSD>::run(ld_n<TI, KSD, STD, LK>(sB, 16 * jt[u], s), ld_n<TI, KSD, STD, LK>(sC, 16 * it[u], s), G[u]);
  }
  f32x4 dC[TT], dB[TT], E[TT], F[TT];
#pragma unroll
  for (int y = 0; y < TT; ++y) dC[y] = dB[y] = f32x4{0.f, 0.f, 0.f, 0.f};
  float frob = 0.f;

  for (int q = 0; q < pairs; ++q) {
    const int hh = q / a.nslab, slab = q % a.nslab, xb = XB == 2 ? q & 1 : 0, hb = hh % HB;
    const TI *sX = sXY[xb][0], *sY = sXY[xb][1];
    if (slab == 0) {
      frob = 0.f;
#pragma unroll
      for (int y = 0; y < TT; ++y) E[y] = F[y] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int u = 0; u < 2; ++u) Q[u] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
    if (q + 1 < pairs) load_rows(q + 1);
#pragma unroll
    for (int s = 0; s < NSC; ++s) {
      FragT<TI, KSC> fs[NS], fd[NS];
#pragma unroll
      for (int j = 0; j < KE; ++j) frob += rs[s][j] * rd[s][j];
      split_frag<TI, KSC, NS>(rs[s], fs);
      split_frag<TI, KSC, NS>(rd[s], fd);
      if (q + 1 < pairs) load_state(q + 1, s);
      if (!mine) continue;
#pragma unroll
      for (int y = 0; y < TT; ++y) {
        const FragT<TI, KSC> yf = ld_n<TI, KSC, STD, LX>(sY, 16 * (ttile0 + y), s);
        const FragT<TI, KSC> xf = ld_n<TI, KSC, STD, LX>(sX, 16 * (ttile0 + y), s);
#pragma unroll
        for (int m = NS - 1; m >= 0; --m) {
          E[y] = Mf<TI, KSC>::run(fs[m], yf, E[y]);
          F[y] = Mf<TI, KSC>::run(fd[m], xf, F[y]);
        }
      }
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      if (w + 8 * u >= 10) continue;
#pragma unroll
      for (int s = 0; s < NSC; ++s)
        Q[u] = Mf<TI, KSC>::run(ld_n<TI, KSC, STD, LX>(sX, 16 * jt[u], s), ld_n<TI, KSC, STD, LX>(sY, 16 * it[u], s), Q[u]);
    }
    if (slab == a.nslab - 1) {
      const float(*gt)[SC] = sh[(hh / HB) & 1][hb];
      float dd = 0.f;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        if (w + 8 * u >= 10) continue;
        const int i = 16 * it[u] + r, j0 = 16 * jt[u] + 4 * g;
        const float ih = gt[0][i], il = gt[1][i];
        const f32x4 jh = ld4(&gt[0][j0]), jl = ld4(&gt[1][j0]), st = ld4(&gt[2][j0]);
        const bool diag = it[u] == jt[u];  // (wave-uniform; below it every pair is in)
        f32x4 wv;
        float row = 0.f, dg = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float gq = __builtin_amdgcn_exp2f((ih - jh[e]) + (il - jl[e])) * Q[u][e];
          if (diag) gq = i >= j0 + e ? gq : 0.f;
          R[u][e] += gq * st[e];
          wv[e] = gq * G[u][e];
          if (diag) {
            dd += i == j0 + e ? Q[u][e] : 0.f;
            dg = i == j0 + e ? wv[e] : dg;
            wv[e] = i == j0 + e ? 0.f : wv[e];
          }
          row += wv[e] * st[e];
        }
        if (diag && (r >> 2) == g) sdiag[hb][i] = dg;
        row = group4_sum(row);
        // column sums over the tile's 16 lanes, four columns side by side
#pragma unroll
        for (int e = 0; e < 4; ++e) wv[e] += dpp<0xB1>(wv[e]);
#pragma unroll
        for (int e = 0; e < 4; ++e) wv[e] += dpp<0x4E>(wv[e]);
#pragma unroll
        for (int e = 0; e < 4; ++e) wv[e] += dpp<0x141>(wv[e]);
#pragma unroll
        for (int e = 0; e < 4; ++e) wv[e] += dpp<0x140>(wv[e]);
        if (r == 0) *reinterpret_cast<f32x4*>(&scol[hb][w + 8 * u][4 * g]) = wv;
        if (g == 0) srow[hb][w + 8 * u][r] = row;
      }
      if (mine) {
#pragma unroll
        for (int y = 0; y < TT; ++y) {
          const int t = 16 * (ttile0 + y) + r, d0 = 16 * dtile + 4 * g;
          const float eb = gt[3][t], ed = gt[4][t] * gt[2][t];
          const f32x4 cv = ld4<TI>(sC + LK::at(t, d0)), bv = ld4<TI>(sB + LK::at(t, d0));
          float ce = cv[0] * E[y][0], bf = bv[0] * F[y][0];
#pragma unroll
          for (int e = 1; e < 4; ++e) {
            ce += cv[e] * E[y][e];
            bf += bv[e] * F[y][e];
          }
          dC[y] += eb * E[y];
          dB[y] += ed * F[y];
          ce = group4_sum(ce);
          bf = group4_sum(bf);
          if (g == 0) {
            sE[hb][w][t] = ce;
            sF[hb][w][t] = bf;
          }
        }
      }
      const float fsum = wave_sum(frob), dsum = wave_sum(dd);
      if (l == 0) {
        sfr[hb][w] = mine && ttile0 == 0 ? fsum : 0.f;  // (each row of the states once)
        sdd[hb][w] = dsum;
      }
      if (hb == HB - 1 || hh == nhd - 1) {
        lds_barrier();  // the batch's sums are complete
        const int h0 = hh - hb;
        if (w <= hb) {  // one head, one token per lane
          const int h = hd0 + h0 + w, ti = l >> 4, b = (h0 / HB) & 1;
          const float(*gw)[SC] = sh[b][w];
          // Pairs (i, j) on both sides of t, by tiles of 16: those of t's own tile as a difference of row
          // and column sums over that tile alone, the others as sums of what is on the far side (over
          // the whole chunk the difference's rounding was common to the chunk's tokens and drowned da_log).
          const int dg = ti * (ti + 1) / 2 + ti;
          float rowo = 0.f, colo = 0.f, ce = 0.f, bf = 0.f, fr = 0.f, dsum8 = 0.f;
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            if (x < ti) rowo += srow[w][ti * (ti + 1) / 2 + x][r];
            if (x > ti) colo += scol[w][x * (x + 1) / 2 + ti][r];
          }
          const float s20 = row16_sum(srow[w][3][r]), s30 = row16_sum(srow[w][6][r]), s31 = row16_sum(srow[w][7][r]);
#pragma unroll
          for (int x = 0; x < 8; ++x) {
            ce += sE[w][x][l];
            bf += sF[w][x][l];
            fr += sfr[w][x];
            dsum8 += sdd[w][x];
          }
          const float step = gw[2][l], z = gw[5][l];
          ce *= gw[3][l];
          bf *= gw[4][l];
          const float cold = scol[w][dg][r], col = cold + colo;
          float suf = rowo + srow[w][dg][r] - step * cold;  // over the tile's tokens from t on
          suf += dpp<0x101>(suf);
          suf += dpp<0x102>(suf);
          suf += dpp<0x104>(suf);
          suf += dpp<0x108>(suf);
          float pre = step * colo;  // over the tile's tokens before t
          pre += dpp<0x111>(pre);
          pre += dpp<0x112>(pre);
          pre += dpp<0x114>(pre);
          pre += dpp<0x118>(pre);
          pre = dpp<0x111>(pre);
          const float far = ti == 1 ? s20 + s30 : ti == 2 ? s30 + s31 : 0.f;  // tiles on either side
          const float before = __shfl_up(wave_scan_incl(step * bf), 1);  // (the last token's own term carries no decay)
          float qt = suf + pre + far + wave_rscan_incl(ce) + (l > 0 ? before : 0.f) + sbn[b][w] * fr;
          const float na = -decay_rate(p.a_log[h]);
          if (na * step < -104.f) qt = 0.f;  // a decay of 2^-150: q holds rounding only, which a large rate would show
          const bool live = l < len;
          const float ddt = live ? (sdiag[w][l] + col + bf + na * qt) / (1.f + expf(-z)) : 0.f;
          if (live) p.ddt[(t0 + l) * p.Hv + h] = ddt;
          const float da = wave_sum(live ? qt * step * na : 0.f), db = wave_sum(ddt);
          if (l == 0) {
            const int64_t at = slot * p.Hv + h, plane = a.slots * p.Hv;
            a.part[at] = da;
            a.part[plane + at] = db;
            a.part[2 * plane + at] = dsum8;
          }
        }
        if (hh + 1 < nhd) {
          gates(hh + 1);
          load_dt(hh + 1 + HB);
        }
      }
    }
    if (q + 1 < pairs) {
      if constexpr (XB == 1) lds_barrier();  // x and dy are used up
      rx.store(sXY[XB == 2 ? xb ^ 1 : 0][0]);
      ry.store(sXY[XB == 2 ? xb ^ 1 : 0][1]);
      lds_barrier();  // the next step's rows (and gates) are in LDS, the sums of this batch are free
    }
  }
  // the heads' sum of Gamma D Q, and its products with b and c
#pragma unroll
  for (int u = 0; u < 2; ++u)
    if (w + 8 * u < 10) {
      f32x4 rest = R[u];
#pragma unroll
      for (int m = 0; m < NR; ++m) {
        TI* at = sR[m] + LX::at(16 * it[u] + r, 16 * jt[u] + 4 * g);
        st4<TI>(at, rest);
#pragma unroll
        for (int e = 0; e < 4; ++e) rest[e] -= (float)(TI)rest[e];
      }
    }
  lds_barrier();
  if (!mine) return;
#pragma unroll
  for (int s = 0; s < NSC; ++s) {
    const FragT<TI, KSC> bf = ld_t<TI, KSC, STD, LK>(sB, 16 * dtile, s), cf = ld_t<TI, KSC, STD, LK>(sC, 16 * dtile, s);
#pragma unroll
    for (int y = 0; y < TT; ++y) {
#pragma unroll
      for (int m = NR - 1; m >= 0; --m) {
        dC[y] = Mf<TI, KSC>::run(bf, ld_n<TI, KSC, STD, LX>(sR[m], 16 * (ttile0 + y), s), dC[y]);
        dB[y] = Mf<TI, KSC>::run(cf, ld_t<TI, KSC, STD, LX>(sR[m], 16 * (ttile0 + y), s), dB[y]);
      }
    }
  }
#pragma unroll
  for (int y = 0; y < TT; ++y) {
    const int t = 16 * (ttile0 + y) + r, d0 = kh * DK + 16 * dtile + 4 * g;
    if (t >= len) continue;
    if (a.parts > 1) {
      float* f = a.fold + ((int64_t)pt * p.T_total + t0 + t) * (p.Hk * DK) + d0;
      st4<float>(f, dC[y]);
      st4<float>(f + (int64_t)a.parts * p.T_total * (p.Hk * DK), dB[y]);
      continue;
    }
    st4<TI>((TI*)p.dc + (t0 + t) * p.dc_rs + d0, dC[y]);
    st4<TI>((TI*)p.db + (t0 + t) * p.db_rs + d0, dB[y]);
  }
}

// dc and db of a chunk and group as the sum of the group's parts, in order, rounded once. Few bytes, bound
// by latency: a thread takes four values, the parts' loads side by side. The first workgroups, 16 heads
// each, do what k_colsum does for longer columns (a launch of its own took 5 us).
template <typename TI> __global__ __launch_bounds__(256) void k_ssm_fold(GradArgs a, ColsumOut sums, int heads) {
  const SsmArgs& p = a.p;
  if ((int)blockIdx.x < 3 * heads) {
    __shared__ double acc[16][17];
    const int plane = (int)blockIdx.x / heads, c = threadIdx.x & 15, k = threadIdx.x >> 4;
    const int h = (int)blockIdx.x % heads * 16 + c;
    const float* in = a.part + (int64_t)plane * a.slots * p.Hv;
    double s = 0.0;
    if (h < p.Hv) {
#pragma unroll 8
      for (int64_t r = k; r < a.slots; r += 16) s += (double)in[r * p.Hv + h];
    }
    acc[k][c] = s;
    __syncthreads();
    if (k == 0 && h < p.Hv && sums.p[plane]) {
#pragma unroll
      for (int i = 1; i < 16; ++i) s += acc[i][c];
      sums.p[plane][h] = (float)s;
    }
    return;
  }
  const int per = p.Dk / 16, kw = p.Hk * p.Dk, cpr = p.Dk / 4;
  const int x = (int)blockIdx.x - 3 * heads, which = x / per & 1, sk = x / (2 * per), kh = sk % p.Hk;
  int64_t t0;
  const int len = slot_chunk(p, sk / p.Hk, t0);
  const float* f = a.fold + (which ? (int64_t)a.parts * p.T_total * kw : 0);
  TI* o = (TI*)(which ? p.db : p.dc);
  const int64_t rs = which ? p.db_rs : p.dc_rs;
  const int i = x % per * 256 + (int)threadIdx.x;
  if (i >= len * cpr) return;
  const int64_t t = t0 + i / cpr;
  const int d = kh * p.Dk + i % cpr * 4;
  f32x4 v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
  for (int q = 0; q < a.parts; ++q) v += ld4<float>(f + ((int64_t)q * p.T_total + t) * kw + d);
  st4<TI>(o + t * rs + d, v);
}

// Workgroups to a group: a chunk's heads are a serial chain, so a short batch's groups are dealt over
// several workgroups (one fits a compute unit) and their dc and db added afterwards. Measured (bf16, heads of
// 128 x 64): 4096 tokens, 32 heads in one group 171 us, in four parts 70 + 6; 8192 tokens, 4 heads in one
// group 36, in two 30 + 6; 512 tokens, 16 heads in one group 83, in 16 parts 18 + 5.
constexpr int kGradGroups = 256;
static int grad_hpp(const SsmArgs& p) {
  const bool packed = p.cu && p.N > 1;  // (a packed batch's lengths are not known here)
  const int64_t chunks = packed ? ssm_slots(p.T_total, p.N) : p.N * (((p.cu ? p.T_total : p.T) + SC - 1) / SC);
  const int64_t groups = chunks * p.Hk;
  int64_t parts = groups > 0 ? kGradGroups / groups : 1;
  if (parts > p.r) parts = p.r;
  return parts > 1 ? (int)((p.r + parts - 1) / parts) : p.r;
}
size_t ssm_fold_bytes(const SsmArgs& p) {
  const int hpp = grad_hpp(p), parts = (p.r + hpp - 1) / hpp;
  return parts > 1 ? (size_t)2 * parts * p.T_total * p.Hk * p.Dk * 4 : 0;
}

template <typename TI> static hipError_t grad_d(const GradArgs& a, hipStream_t s) {
  const unsigned grid = (unsigned)(a.slots * a.p.Hk * a.parts);
  switch (a.p.Dk) {
    case 16: traced("k_ssm_grad", s, [&] { k_ssm_grad<TI, 16><<<grid, 512, 0, s>>>(a); }); break;
    case 32: traced("k_ssm_grad", s, [&] { k_ssm_grad<TI, 32><<<grid, 512, 0, s>>>(a); }); break;
    case 64: traced("k_ssm_grad", s, [&] { k_ssm_grad<TI, 64><<<grid, 512, 0, s>>>(a); }); break;
    case 128: traced("k_ssm_grad", s, [&] { k_ssm_grad<TI, 128><<<grid, 512, 0, s>>>(a); }); break;
    default: return hipErrorInvalidValue;
  }
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const ColsumOut sums{{a.p.da_log, a.p.ddt_bias, a.p.dd_skip}};
  const bool any = a.p.da_log || a.p.ddt_bias || a.p.dd_skip;
  if (a.parts == 1) return any ? launch_colsum(a.part, a.slots, a.p.Hv, sums, 3, s) : hipSuccess;
  const int heads = any ? (a.p.Hv + 15) / 16 : 0;
  const unsigned blocks = (unsigned)(3 * heads + a.slots * a.p.Hk * 2 * (a.p.Dk / 16));
  traced("k_ssm_fold", s, [&] { k_ssm_fold<TI><<<blocks, 256, 0, s>>>(a, sums, heads); });
  return hipGetLastError();
}

hipError_t launch_ssm_grad(const SsmArgs& p, int dtype, const float* ds, float* part, float* fold, hipStream_t s) {
  GradArgs a;
  a.p = p;
  a.sv = p.sv;
  a.ds = ds;
  a.part = part;
  a.fold = fold;
  a.hpp = grad_hpp(p);
  a.parts = (p.r + a.hpp - 1) / a.hpp;
  a.nslab = (p.Dv + SP - 1) / SP;
  a.slots = ssm_slots(p.T_total, p.N);
  return dtype == 0 ? grad_d<float>(a, s) : grad_d<__bf16>(a, s);
}

}  // namespace gdn
