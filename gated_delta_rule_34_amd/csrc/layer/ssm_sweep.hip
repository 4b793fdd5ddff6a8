// ssm_sweep.hip -- the selective state space scan's sweep over a sequence's chunks, on gfx950:
// outputs y and the state going forward in time, or dx and the state's adjoint going backward
// (the formulas stand in ssm_common.h).
//
// One workgroup per (sequence, segment, head, 64 columns of x): eight waves, wave w with 16 columns
// (w mod 4) and half of the state's rows (w / 4) in its accumulators; columns of the state never mix,
// and the two halves' shares of S^T Q meet in LDS. Per chunk the products K Q^T, S^T Q, K^T (w X) and
// M X run on the matrix cores; every product is formed transposed, so that a lane holds four adjacent
// columns of one token. M and the state enter the products of an output as two bfloat16 terms each, so that a
// row carries no rounding but its own (as one term each, whose rounding does not shrink where a row's terms
// cancel, y and dx were 1.9e-3 off the 64-bit result instead of 1.66e-3, for 5% less time). The next chunk's
// rows are in registers while a chunk is computed. A chunk is a chain of short dependent products with three
// barriers. Eight waves of 128 registers and 81 KB of LDS let two workgroups (four waves per SIMD) share
// a compute unit where there are that many. Measured (bf16, 4 x 4096 tokens, 64 heads of 128 x 64 in 8 groups,
// which is one workgroup to a compute unit): 264 us without and 298 us with saved states (0.54 GB more written),
// 300 us in reverse; the rows alone would take a copy 66 us. A chunk takes a workgroup some 9000 cycles.
//
// Few sequences and heads leave compute units idle over a long serial chain, so a sequence is then
// cut into S segments: a first launch runs the state alone over all segments but the last, from
// zero, and the second starts each segment from the earlier segments' states and decays (16384 tokens, 32 heads in one group:
// 49 us for the states, 109 us for the outputs).
#include "ssm_common.h"

namespace gdn {

struct SweepArgs {
  int N, Hk, Hv, r, Dv, nslab, S, T, xcd;
  int64_t T_total;
  const int* cu;
  const void *k, *q, *x;  // the vectors that write and that read the state, the values
  int64_t k_rs, q_rs, x_rs, o_rs;
  void* o;
  const float *dt, *a_log, *dt_bias, *d_skip;
  const float* s0;  // [N][Hv][Dk][Dv] or nullptr
  float* st;        // final state, or nullptr
  float* sv;        // the state before each chunk [slot][Hv][Dk][Dv], or nullptr
  float* loc;       // segments' states from zero, in the accumulators' order
  float* dec;       // [N][S][Hv] decay over each segment
};

// Gate rows in LDS: gamma and its remainder, the step (the weight of an input, in reverse of an
// output), the decays with which a token reads and writes the state.
enum { G_HI, G_LO, G_IN, G_RD, G_WR, G_ROWS };

constexpr int kMinChunks = 2;  // least chunks of a segment

template <typename TI, int DK> constexpr int sweep_waves() { return sizeof(TI) == 4 ? 2 : 4; }  // per SIMD

template <typename TI, int DK, bool REV, bool OUT>
__global__ __launch_bounds__(512, (sweep_waves<TI, DK>())) void k_ssm_sweep(SweepArgs a) {
  constexpr int NT = 512, DH = DK >= 32 ? DK / 2 : 16, ND = DH / 16;  // this wave's rows of the state
  constexpr int KSD = ks_of<TI, DK>(), NSD = DK / KSD, KSC = ks_of<TI, SC>(), NSC = SC / KSC;
  constexpr int KSH = ks_of<TI, DH>(), NSH = DH / KSH;
  constexpr int NS = ssm_split<TI>(), NO = out_split<TI>(), TRI = REV ? TRI_UP : TRI_LOW, GB = 3, GR = GB + 1;
  using LK = PadRow<TI, DK>;
  using LX = Swz<TI, SP, true>;
  using LM = Swz<TI, SC, false>;
  __shared__ __align__(16) TI sK[LK::size(SC)];
  __shared__ __align__(16) TI sQ[OUT ? LK::size(SC) : 8];
  __shared__ __align__(16) TI sX[SC * SP];
  __shared__ __align__(16) TI sM[OUT ? NO : 1][OUT ? SC * SC : 8];  // M, as NO terms that add up to it
  __shared__ __align__(16) f32x4 sP[OUT ? 8 * 2 * 64 : 1];  // shares of S^T Q for the other half
  __shared__ __align__(16) float sg[GR][G_ROWS][SC];
  __shared__ float sbn[GR];

  const int segs = OUT ? a.S : a.S - 1;
  int grp, mem;
  if (a.xcd) {
    if (!xcd_group(blockIdx.x, a.N * segs * a.Hk, a.r * a.nslab, grp, mem)) return;
  } else {
    grp = blockIdx.x / (a.r * a.nslab);
    mem = blockIdx.x % (a.r * a.nslab);
  }
  const int kh = grp % a.Hk, n = (grp / a.Hk) % a.N, sgm = grp / a.Hk / a.N;
  const int h = kh * a.r + mem / a.nslab, slab = mem % a.nslab;
  const int w = wave_id(), l = lane_id(), g = l >> 4, r = l & 15;
  const int cw = w & 3, hf = w >> 2;            // this wave's columns and half
  const int col0 = slab * SP + 16 * cw;         // its first column of the head
  const bool cols = col0 < a.Dv;                // (a head of 16 or 32 leaves waves without columns)
  const bool has = cols && hf * DH < DK;        // whether it holds a part of the state
  const int d0 = hf * DH + 4 * g;               // its first row there, this lane's
  const int ncols = a.Dv - slab * SP < SP ? a.Dv - slab * SP : SP;

  int64_t lo, hi;
  ssm_seq(a.cu, a.T, a.T_total, n, lo, hi);
  // a short sequence takes fewer segments than the batch has: the workgroups of the others have nothing to do
  const int nch = (int)((hi - lo + SC - 1) / SC), cps = max((nch + a.S - 1) / a.S, kMinChunks);
  const int last = max(nch - 1, 0) / cps;  // the segment with the sequence's end
  if (OUT ? sgm > last : sgm >= last) return;
  const int k0 = sgm * cps, k1 = min(nch, k0 + cps);

  const double neg_a = neg_a_log2(a.a_log[h]);
  const float bias = a.dt_bias ? a.dt_bias[h] : 0.f;
  const float dsk = a.d_skip ? a.d_skip[h] : 0.f;
  const TI* kp = (const TI*)a.k + kh * DK;
  const TI* qp = (const TI*)a.q + kh * DK;
  const TI* xp = (const TI*)a.x + (int64_t)h * a.Dv + slab * SP;

  auto chunk = [&](int k) { return REV ? nch - 1 - k : k; };
  auto clen = [&](int c) { const int64_t rest = hi - lo - (int64_t)c * SC; return (int)(rest < SC ? rest : SC); };
  TileRegs<TI, DK, LK, NT> rk, rq;
  TileRegs<TI, SP, LX, NT> rx;
  rk.init(a.k_rs, DK);
  if constexpr (OUT) rq.init(a.q_rs, DK);
  rx.init(a.x_rs, ncols);
  const uint32_t orow = (uint32_t)a.o_rs * (uint32_t)sizeof(TI);
  // Gates come GB chunks at a time, one for each of GB waves: a chunk's are a long chain of dependent
  // operations that by one wave in every chunk took a fifth of the step (every third chunk takes 4% less than
  // every second one: 4 x 4096 tokens, 64 heads). A ring of GB + 1 holds them: the chunk in work keeps its own.
  float rdt = 0.f;  // dt of this wave's chunk of the next ones
  auto load = [&](int k) {
    const int c = chunk(k), len = clen(c);
    const int64_t t0 = lo + (int64_t)c * SC;
    rk.template load<false>(kp + t0 * a.k_rs, len);
    if constexpr (OUT) rq.template load<false>(qp + t0 * a.q_rs, len);
    rx.template load<true>(xp + t0 * a.x_rs, len);
  };
  auto load_dt = [&](int k) {
    const int c = chunk(k);
    rdt = w < GB && k < k1 && l < clen(c) ? a.dt[(lo + (int64_t)c * SC + l) * a.Hv + h] : 0.f;
  };
  auto gates = [&](int k) {
    if (w >= GB) return;
    const bool valid = k < k1 && l < clen(chunk(k));
    const Gate q = chunk_gate(rdt, bias, neg_a, valid);
    const float hi32 = (float)q.gam, eb = exp2_d(q.gam), ee = exp2_d(q.tot - q.gam);
    float(*gt)[SC] = sg[(k - k0) & (GR - 1)];
    gt[G_HI][l] = hi32;
    gt[G_LO][l] = (float)(q.gam - (double)hi32);
    gt[G_IN][l] = q.step;
    gt[G_RD][l] = REV ? ee : eb;
    gt[G_WR][l] = REV ? (valid ? eb : 0.f) : ee * q.step;
    if (l == 63) sbn[(k - k0) & (GR - 1)] = exp2_d(q.tot);
  };
  if (k0 < k1) {
    load_dt(k0 + w);
    load(k0);
  }

  // the state: tile t holds rows d0 + 16 t + e of column col0 + r
  f32x4 S[ND];
#pragma unroll
  for (int t = 0; t < ND; ++t) S[t] = f32x4{0.f, 0.f, 0.f, 0.f};
  const int64_t nh = (int64_t)n * a.Hv + h;
  if constexpr (OUT) {
    if (a.s0 && has) {
      const float* s0 = a.s0 + nh * DK * a.Dv + col0 + r;
#pragma unroll
      for (int t = 0; t < ND; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) S[t][e] = s0[(int64_t)(d0 + 16 * t + e) * a.Dv];
    }
    for (int j = 0; j < sgm; ++j) {
      const int64_t nj = ((int64_t)n * a.S + j) * a.Hv + h;
      const float d = a.dec[nj];
      const f32x4* p = reinterpret_cast<const f32x4*>(a.loc) + ((nj * a.nslab + slab) * ND) * NT + threadIdx.x;
#pragma unroll
      for (int t = 0; t < ND; ++t) S[t] = d * S[t] + p[t * NT];
    }
    for (int i = threadIdx.x; i < NO * SC * SC; i += NT) sM[0][i] = (TI)0.f;  // the tiles past the diagonal stay zero
  }
  float dec = 1.f;
  auto put = [&](float* st) {  // the state as [Dk][Dv] of one head
    const __amdgpu_buffer_rsrc_t rs = rows_rsrc(st, DK * a.Dv * 4);
    const uint32_t voff = (uint32_t)(d0 * a.Dv + col0 + r) * 4u;
#pragma unroll
    for (int t = 0; t < ND; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float v = S[t][e];
        __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v), rs, (int)voff, (16 * t + e) * a.Dv * 4, 0);
      }
  };
  auto save = [&](int k) {  // the state before chunk k
    put(a.sv + ((lo / SC + n + chunk(k)) * a.Hv + h) * (int64_t)DK * a.Dv);
  };

  if (k0 < k1) {
    if (OUT && a.sv && has) save(k0);
    gates(k0 + w);
    load_dt(k0 + GB + w);
    rk.store(sK);
    if constexpr (OUT) rq.store(sQ);
    rx.store(sX);
  }
  for (int k = k0; k < k1; ++k) {
    const int c = chunk(k), len = clen(c);
    const int64_t t0 = lo + (int64_t)c * SC;
    lds_barrier();  // the chunk's rows and gates are in LDS, M and the shares are free
    if (k + 1 < k1) load(k + 1);
    const float(*gt)[SC] = sg[(k - k0) & (GR - 1)];
    const float bn = sbn[(k - k0) & (GR - 1)];
    f32x4 o[4];
    if constexpr (OUT) {
      // M = Gamma o (Q K^T) o inputs' weights: its ten tiles dealt over the waves
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int idx = w + 8 * u;
        if (idx >= 10) continue;
        const int big = idx >= 6 ? 3 : idx >= 3 ? 2 : idx >= 1 ? 1 : 0, small = idx - big * (big + 1) / 2;
        const int it = REV ? small : big, jt = REV ? big : small;
        f32x4 m = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = 0; s < NSD; ++s)
          m = Mf<TI, KSD>::run(ld_n<TI, KSD, STD, LK>(sK, 16 * jt, s), ld_n<TI, KSD, STD, LK>(sQ, 16 * it, s), m);
        const int i = 16 * it + r, j0 = 16 * jt + 4 * g;
        const float ih = gt[G_HI][i], il = gt[G_LO][i];
        const f32x4 jh = ld4(&gt[G_HI][j0]), jl = ld4(&gt[G_LO][j0]), wi = ld4(&gt[G_IN][j0]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float d = REV ? (jh[e] - ih) + (jl[e] - il) : (ih - jh[e]) + (il - jl[e]);
          const bool in = REV ? i <= j0 + e : i >= j0 + e;
          m[e] *= __builtin_amdgcn_exp2f(d);
          if constexpr (!REV) m[e] *= wi[e];
          m[e] = in ? m[e] : 0.f;
        }
#pragma unroll
        for (int q = 0; q < NO; ++q) {
          st4<TI>(sM[q] + LM::at(i, j0), m);
          if (q + 1 < NO) {
#pragma unroll
            for (int e = 0; e < 4; ++e) m[e] -= (float)(TI)m[e];
          }
        }
      }
      // this half's share of S^T Q, decayed; two token tiles of it go to the other half
#pragma unroll
      for (int t = 0; t < 4; ++t) o[t] = f32x4{0.f, 0.f, 0.f, 0.f};
      if (has) {
#pragma unroll
        for (int s = 0; s < NSH; ++s) {
          FragT<TI, KSH> sf[NO];
          acc_split<TI, KSH, NO>(S, s, sf);
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            const FragT<TI, KSH> qf = ld_n<TI, KSH, ACC, LK>(sQ, 16 * t, hf * NSH + s);
#pragma unroll
            for (int m = NO - 1; m >= 0; --m) o[t] = Mf<TI, KSH>::run(sf[m], qf, o[t]);
          }
        }
      }
      if (hf == 0) {
        sP[(w * 2 + 0) * 64 + l] = o[2];
        sP[(w * 2 + 1) * 64 + l] = o[3];
      } else {
        sP[(w * 2 + 0) * 64 + l] = o[0];
        sP[(w * 2 + 1) * 64 + l] = o[1];
        o[0] = o[2];
        o[1] = o[3];
      }
    }
    FragT<TI, KSC> xf[NSC];
    if (cols) {
#pragma unroll
      for (int s = 0; s < NSC; ++s) xf[s] = ld_t<TI, KSC, STD, LX>(sX, 16 * cw, s);
    }
    if (has) {  // the state past this chunk
#pragma unroll
      for (int t = 0; t < ND; ++t) S[t] *= bn;
#pragma unroll
      for (int s = 0; s < NSC; ++s) {
        FragT<TI, KSC> u[NS];
        scale_split<TI, KSC, NS>(xf[s], gt[G_WR], s, u);
#pragma unroll
        for (int t = 0; t < ND; ++t) {
          const FragT<TI, KSC> kf = ld_t<TI, KSC, STD, LK>(sK, hf * DH + 16 * t, s);
#pragma unroll
          for (int m = NS - 1; m >= 0; --m) S[t] = Mf<TI, KSC>::run(kf, u[m], S[t]);
        }
      }
    }
    dec *= bn;
    lds_barrier();  // M and the shares are complete, K and Q are free
    if constexpr (OUT) {
      if (a.sv && has && k + 1 < k1) save(k + 1);
      if (cols) {  // this wave's token tiles 2 hf and 2 hf + 1
        const __amdgpu_buffer_rsrc_t rs = rows_rsrc((TI*)a.o + t0 * a.o_rs + (int64_t)h * a.Dv, (uint32_t)len * orow);
#pragma unroll
        for (int t = 0; t < 2; ++t) o[t] = (o[t] + sP[((w ^ 4) * 2 + t) * 64 + l]) * gt[G_RD][32 * hf + 16 * t + r];
        // steps of M X whose tiles are all zero are left out (wave-uniform)
#pragma unroll
        for (int s = 0; s < NSC; ++s)
#pragma unroll
          for (int t = 0; t < 2; ++t)
            if (hf == 0 ? !tri_skip<TRI, KSC>(s, t) : !tri_skip<TRI, KSC>(s, 2 + t)) {
#pragma unroll
              for (int m = NO - 1; m >= 0; --m)
                o[t] = Mf<TI, KSC>::run(xf[s], ld_n<TI, KSC, STD, LM>(sM[m], 32 * hf + 16 * t, s), o[t]);
            }
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const int i = 32 * hf + 16 * t + r;  // (rows past the chunk's end are dropped)
          f32x4 v = o[t];
          if constexpr (REV) v *= gt[G_IN][i];
          buf_st4<TI>(rs, (uint32_t)i * orow + (uint32_t)(col0 + 4 * g) * (uint32_t)sizeof(TI),
                      v + dsk * ld4<TI>(sX + LX::at(i, 16 * cw + 4 * g)));
        }
      }
    }
    if (k + 1 < k1) {
      if ((k + 1 - k0) % GB == 0) {  // the next chunks' gates
        gates(k + 1 + w);
        load_dt(k + 1 + GB + w);
      }
      rk.store(sK);
      if constexpr (OUT) {
        rq.store(sQ);
        lds_barrier();  // X and M are used up
      }
      rx.store(sX);
    }
  }
  if constexpr (OUT) {
    if (a.st && has && sgm == last) put(a.st + nh * DK * a.Dv);
  } else {
    const int64_t nj = ((int64_t)n * a.S + sgm) * a.Hv + h;
    f32x4* p = reinterpret_cast<f32x4*>(a.loc) + ((nj * a.nslab + slab) * ND) * NT + threadIdx.x;
#pragma unroll
    for (int t = 0; t < ND; ++t) p[t * NT] = S[t];
    if (slab == 0 && threadIdx.x == 0) a.dec[nj] = dec;
  }
}

// Segments per sequence: two workgroups to a compute unit, at most one for every kMinChunks chunks of the
// longest sequence there can be. A segment costs its states and a second read of its rows, so two gain
// nothing (4 x 4096 tokens, 64 heads: one segment 263 us, two 261), more do (16384 tokens, 32 heads: 8 of
// them 187 us, 16 of them 151, 32 of them 202; 300 tokens, 8 heads: one 23, three 20). A packed batch's lengths
// are not known here: its short sequences leave their further segments empty (lengths up to 777, 6 heads of
// 32 x 32, float32, training step: three segments 98 us, seven 68; 16 x 512 tokens, 4 heads: one 35 us, four 26; 3000, 1000
// and 200 tokens, 32 heads: one 169, three 94, five 77). A float32 workgroup with a state of 128 rows has its compute unit
// to itself, so that the rule cuts such sequences finer than is best: 2048 tokens, 32 heads of 128 x 64 in 16 segments 77 us,
// in 8 of them 70 (training step 294 and 278).
constexpr int kWantGroups = 512, kMaxSegments = 32;
static int ssm_segments(const SsmArgs& a) {
  if (a.N == 0) return 1;
  const int64_t groups = (int64_t)a.N * a.Hv * ((a.Dv + SP - 1) / SP);
  const int64_t longest = ((a.cu ? a.T_total : a.T) + SC - 1) / SC, most = (longest + kMinChunks - 1) / kMinChunks;
  int64_t s = kWantGroups / groups;
  if (s > most) s = most;
  if (s > kMaxSegments) s = kMaxSegments;
  return s <= 2 ? 1 : (int)s;
}

static size_t up256(size_t x) { return (x + 255) / 256 * 256; }
static size_t seg_bytes(const SsmArgs& a) {
  const int S = ssm_segments(a);
  if (S == 1) return 0;
  const size_t u = (size_t)a.N * S * a.Hv;
  return up256(u * ((a.Dv + SP - 1) / SP) * (a.Dk < 32 ? 32 : a.Dk) * SP * 4) + up256(u * 4);
}
size_t ssm_saved_bytes(const SsmArgs& a) { return (size_t)ssm_slots(a.T_total, a.N) * a.Hv * a.Dk * a.Dv * 4; }
size_t ssm_fwd_ws_bytes(const SsmArgs& a) { return seg_bytes(a); }

template <typename TI, int DK, bool REV> static hipError_t sweep_go(const SsmArgs& a, float* sv, float* seg, hipStream_t s) {
  SweepArgs v{};
  v.N = a.N; v.Hk = a.Hk; v.Hv = a.Hv; v.r = a.r; v.Dv = a.Dv; v.T = a.T; v.T_total = a.T_total; v.cu = a.cu;
  v.nslab = (a.Dv + SP - 1) / SP;
  v.S = ssm_segments(a);
  v.k = REV ? a.c : a.b; v.k_rs = REV ? a.c_rs : a.b_rs;
  v.q = REV ? a.b : a.c; v.q_rs = REV ? a.b_rs : a.c_rs;
  v.x = REV ? a.dy : a.x; v.x_rs = REV ? a.dy_rs : a.x_rs;
  v.o = REV ? a.dx : a.y; v.o_rs = REV ? a.dx_rs : a.y_rs;
  v.dt = a.dt; v.a_log = a.a_log; v.dt_bias = a.dt_bias; v.d_skip = a.d_skip;
  v.s0 = REV ? a.dST : a.S0;
  v.st = REV ? a.dS0 : a.ST;
  v.sv = sv;
  v.loc = seg;
  v.dec = seg + (v.S > 1 ? up256((size_t)a.N * v.S * a.Hv * v.nslab * (DK < 32 ? 32 : DK) * SP * 4) / 4 : 0);
  // A group's heads share b and c: with many groups they go to one XCD (workgroups are dealt to
  // the eight XCDs in turn) and share its L2; few groups would leave XCDs idle. A packed batch's segments
  // are dealt one by one: a long sequence's would else meet on a few compute units (1500, 20, 300, 44, 5
  // and 700 tokens, 24 heads: 50 us, so 39). Later segments come last, the empty ones behind the others.
  auto grid = [&](int segs) {
    const int G = a.N * segs * a.Hk, m = a.r * v.nslab;
    v.xcd = G >= 32 && !(v.S > 1 && a.cu && a.N > 1);
    return v.xcd ? xcd_grid(G, m) : G * m;
  };
  if (v.S > 1) {
    const int b = grid(v.S - 1);
    traced(REV ? "k_ssm_state_rev" : "k_ssm_state", s, [&] { k_ssm_sweep<TI, DK, REV, false><<<b, 512, 0, s>>>(v); });
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  const int b = grid(v.S);
  traced(REV ? "k_ssm_sweep_rev" : "k_ssm_sweep", s, [&] { k_ssm_sweep<TI, DK, REV, true><<<b, 512, 0, s>>>(v); });
  return hipGetLastError();
}

template <typename TI, bool REV> static hipError_t sweep_d(const SsmArgs& a, float* sv, float* seg, hipStream_t s) {
  switch (a.Dk) {
    case 16: return sweep_go<TI, 16, REV>(a, sv, seg, s);
    case 32: return sweep_go<TI, 32, REV>(a, sv, seg, s);
    case 64: return sweep_go<TI, 64, REV>(a, sv, seg, s);
    case 128: return sweep_go<TI, 128, REV>(a, sv, seg, s);
  }
  return hipErrorInvalidValue;
}

hipError_t launch_ssm_forward(const SsmArgs& a, int dtype, hipStream_t s) {
  return dtype == 0 ? sweep_d<float, false>(a, a.sv, a.ws, s) : sweep_d<__bf16, false>(a, a.sv, a.ws, s);
}

// Backward workspace: the adjoints at the chunks' ends, the parameters' partials, the groups' parts, the segments.
size_t ssm_bwd_ws_bytes(const SsmArgs& a) {
  return up256(ssm_saved_bytes(a)) + up256((size_t)ssm_slots(a.T_total, a.N) * 3 * a.Hv * 4) + up256(ssm_fold_bytes(a)) + seg_bytes(a);
}

hipError_t launch_ssm_backward(const SsmArgs& a, int dtype, hipStream_t s) {
  float* ds = a.ws;
  float* part = ds + up256(ssm_saved_bytes(a)) / 4;
  float* fold = part + up256((size_t)ssm_slots(a.T_total, a.N) * 3 * a.Hv * 4) / 4;
  float* seg = fold + up256(ssm_fold_bytes(a)) / 4;
  hipError_t e = hipSuccess;
  if (a.N > 0) {
    e = dtype == 0 ? sweep_d<float, true>(a, ds, seg, s) : sweep_d<__bf16, true>(a, ds, seg, s);
    return e == hipSuccess ? launch_ssm_grad(a, dtype, ds, part, fold, s) : e;
  }
  if (a.da_log || a.ddt_bias || a.dd_skip)  // nothing to sum
    e = launch_colsum(part, 0, a.Hv, ColsumOut{{a.da_log, a.ddt_bias, a.dd_skip}}, 3, s);
  return e;
}

}  // namespace gdn
