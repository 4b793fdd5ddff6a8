// paged_attn.hip -- attention of one new token per sequence over a paged cache, on gfx950.
//
//   z_t = scale q . k_t,  out = sum_t exp(z_t - lse) v_t,  lse = log sum_t exp(z_t)
//
// One pass over the cache with the running maximum m and sum l of the softmax, in log2 units. Every key and value is
// read once: bound by HBM. A workgroup takes a chunk of one sequence's tokens for up to 16 query heads of a key head,
// its waves tiles of 16 tokens in turn. Nothing passes through LDS inside a tile:
//   S = K Q^T with the tokens as rows (16x16x32 bf16, or 16x16x4 float32): lane (g, j) = (l / 16, l % 16) reads 16 bytes of
//   token j as its operand and receives S of tokens 4g .. 4g + 3 for head j;
//   O += P V by 16x16x4 float32 instructions, step i over the tokens 4g + i: P's operand is the very register that S left
//   in the lane, V's a piece of token 4g + i's row, whose columns the accumulators take in the order in which they are
//   read. So P keeps its 32 bits, and V is read as whole rows.
// The maximum only moves (and O is only rescaled) when a score exceeds it by 2^8 in weight. Waves join in LDS, chunks in a second
// launch, in a fixed order.
#include "../gdn_common.h"
#include "../layer/vec8.h"
#include "hybrid_internal.h"

namespace gdn {

constexpr int PW = 4;        // waves per workgroup
constexpr int PT = 16;       // tokens per tile
constexpr float kNone = -__builtin_inff();

// What a sequence's length and window leave: tokens [lo, len), chunks from `base` on.
struct PagedSpan {
  int lo, len, base, chunks;
};
__device__ __forceinline__ PagedSpan paged_span(const PagedArgs& a, int n, int chunk) {
  PagedSpan s;
  int len = a.lens[n];
  s.len = len < 0 ? 0 : len > a.max_len ? a.max_len : len;
  s.lo = a.window > 0 && s.len > a.window ? s.len - a.window : 0;
  s.base = s.lo & ~(PT - 1);
  s.chunks = (s.len - s.base + chunk - 1) / chunk;
  return s;
}

// A lane's pieces of one key (KP of 16 bytes) and of one value row (VP pieces of PE values: D / 16 of them).
template <typename TI, int D> struct PagedTile {
  static constexpr int KP = D / (64 / (int)sizeof(TI));
  static constexpr int VE = D / 16, PE = VE < 16 / (int)sizeof(TI) ? VE : 16 / (int)sizeof(TI), VP = VE / PE;
  static constexpr int W = PE * (int)sizeof(TI) / 4;  // dwords of a piece of V
  typedef int32_t vpiece __attribute__((ext_vector_type(W)));
  i32x4 k[KP];
  vpiece v[4][VP];
  bool full;      // every token counts (wave-uniform)
  uint32_t mask;  // else: bit i: token 4g + i counts
};
template <> struct PagedTile<__bf16, 32> {
  static constexpr int KP = 1, VE = 2, PE = 2, VP = 1, W = 1;
  typedef int32_t vpiece;
  i32x4 k[1];
  int32_t v[4][1];
  bool full;
  uint32_t mask;
};

// Value e of a piece as float32.
template <typename TI, typename P> __device__ __forceinline__ float piece_at(const P& p, int e) {
  uint32_t w;
  if constexpr (sizeof(P) == 4) w = (uint32_t)p;
  else w = (uint32_t)p[sizeof(TI) == 2 ? e / 2 : e];
  if constexpr (sizeof(TI) == 2) w = e & 1 ? w & 0xFFFF0000u : w << 16;
  return __uint_as_float(w);
}

template <typename TI, int D, bool UNI, bool PART>
__global__ __launch_bounds__(64 * PW) void k_paged(PagedArgs a, int chunk, int splits, int gt) {
  typedef PagedTile<TI, D> Tile;
  constexpr int KP = Tile::KP, VE = Tile::VE, PE = Tile::PE, VP = Tile::VP;
  __shared__ __align__(16) float so[PW][8][D];
  __shared__ float sm[PW][16], sl[PW][16];
  int bx = (int)blockIdx.x;
  const int split = bx % splits;
  bx /= splits;
  const int ht = bx % gt;
  bx /= gt;
  const int hk = bx % a.Hk, n = bx / a.Hk;
  const int r = a.Hq / a.Hk, h0 = hk * r + ht * 16, nh = r - ht * 16 < 16 ? r - ht * 16 : 16;
  const PagedSpan sp = paged_span(a, n, chunk);
  if (PART && split >= sp.chunks) return;
  const int w = wave_id(), g = lane_id() >> 4, j = lane_id() & 15;
  const int t0 = sp.base + split * chunk, t1 = t0 + chunk < sp.len ? t0 + chunk : sp.len;
  const TI *kp = (const TI*)a.kp, *vp = (const TI*)a.vp;
  const int* table = a.table + (int64_t)n * a.max_pages;

  i32x4 q[KP];
#pragma unroll
  for (int p = 0; p < KP; ++p) {
    q[p] = i32x4{0, 0, 0, 0};
    if (j < nh) q[p] = *reinterpret_cast<const i32x4*>((const TI*)a.q + (int64_t)n * a.q_rs + (int64_t)(h0 + j) * D + (p * 64 + g * 16) / (int)sizeof(TI));
  }
  const float sc = a.scale * 1.44269504f;
  f32x4 o[VE];
#pragma unroll
  for (int e = 0; e < VE; ++e) o[e] = f32x4{0.f, 0.f, 0.f, 0.f};
  float m = kNone, l = 0.f;  // of head j; l: this lane's tokens only

  // Row of token t among the pool's rows of this key head, or none.
  auto row_of = [&](int t, bool& ok) -> uint32_t {
    const uint32_t pg = (uint32_t)t / (uint32_t)a.page;
    ok = t >= sp.lo && t < t1;
    const int page = ok ? table[pg] : -1;
    ok = page >= 0 && page < a.n_pages;
    return ((uint32_t)page * (uint32_t)a.Hk + (uint32_t)hk) * (uint32_t)a.page + ((uint32_t)t - pg * (uint32_t)a.page);
  };
  auto load_k = [&](Tile& x, const TI* p) {
#pragma unroll
    for (int c = 0; c < KP; ++c) x.k[c] = __builtin_nontemporal_load(reinterpret_cast<const i32x4*>(p + (c * 64 + g * 16) / (int)sizeof(TI)));
  };
  auto load_v = [&](Tile& x, int i, const TI* p) {
#pragma unroll
    for (int c = 0; c < VP; ++c)
      x.v[i][c] = __builtin_nontemporal_load(reinterpret_cast<const typename Tile::vpiece*>(p + c * 16 * PE + j * PE));
  };
  auto load = [&](Tile& x, int t) {
    if constexpr (UNI) {  // a tile lies in one page
      const uint32_t pg = (uint32_t)t / (uint32_t)a.page;
      const int page = __builtin_amdgcn_readfirstlane(table[pg]);
      const bool ok = page >= 0 && page < a.n_pages;
      x.full = ok && t >= sp.lo && t + PT <= t1;
      const int64_t row = ((int64_t)page * a.Hk + hk) * a.page + ((uint32_t)t - pg * (uint32_t)a.page);
      if (x.full) {
        load_k(x, kp + (row + j) * D);
#pragma unroll
        for (int i = 0; i < 4; ++i) load_v(x, i, vp + (row + 4 * g + i) * D);
        return;
      }
      x.mask = 0;
#pragma unroll
      for (int c = 0; c < KP; ++c) x.k[c] = i32x4{0, 0, 0, 0};
      if (ok && t + j >= sp.lo && t + j < t1) load_k(x, kp + (row + j) * D);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int c = 0; c < VP; ++c) x.v[i][c] = typename Tile::vpiece{};
        if (ok && t + 4 * g + i >= sp.lo && t + 4 * g + i < t1) {
          x.mask |= 1u << i;
          load_v(x, i, vp + (row + 4 * g + i) * D);
        }
      }
    } else {
      bool ok;
      const uint32_t row = row_of(t + j, ok);
      const uint64_t all = __ballot(ok);
      x.full = all == ~0ull;
      x.mask = (uint32_t)(all >> (4 * g)) & 15;  // (lanes 0 .. 15 hold the tile's tokens)
#pragma unroll
      for (int c = 0; c < KP; ++c) x.k[c] = i32x4{0, 0, 0, 0};
      if (ok) load_k(x, kp + (int64_t)row * D);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t vrow = (uint32_t)__builtin_amdgcn_ds_bpermute((4 * g + i) << 2, (int)row);
#pragma unroll
        for (int c = 0; c < VP; ++c) x.v[i][c] = typename Tile::vpiece{};
        if (x.mask >> i & 1) load_v(x, i, vp + (int64_t)vrow * D);
      }
    }
  };
  auto use = [&](const Tile& x) {
    f32x4 s{0.f, 0.f, 0.f, 0.f};
    if constexpr (sizeof(TI) == 2) {
#pragma unroll
      for (int c = 0; c < KP; ++c)
        s = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, x.k[c]), __builtin_bit_cast(bf16x8, q[c]), s, 0, 0, 0);
    } else {
#pragma unroll
      for (int c = 0; c < KP; ++c)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          s = __builtin_amdgcn_mfma_f32_16x16x4f32(__int_as_float(x.k[c][e]), __int_as_float(q[c][e]), s, 0, 0, 0);
    }
    float z[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      z[i] = s[i] * sc;
      if (!x.full && !(x.mask >> i & 1)) z[i] = kNone;
    }
    const float top = fmaxf(fmaxf(z[0], z[1]), fmaxf(z[2], z[3]));
    if (__any(top > m + 8.f)) {  // (the first score exceeds any)
      float mx = fmaxf(top, m);
      mx = fmaxf(mx, __shfl_xor(mx, 16));
      mx = fmaxf(mx, __shfl_xor(mx, 32));
      const float f = m == kNone ? 0.f : __builtin_amdgcn_exp2f(m - mx);  // (m is none: nothing there to scale)
      m = mx;
      l *= f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float fo = __shfl(f, 4 * g + i);
#pragma unroll
        for (int e = 0; e < VE; ++e) o[e][i] *= fo;
      }
    }
    const float ref = m == kNone ? 0.f : m;
    float p[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      p[i] = __builtin_amdgcn_exp2f(z[i] - ref);
      l += p[i];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int e = 0; e < VE; ++e)
        o[e] = __builtin_amdgcn_mfma_f32_16x16x4f32(p[i], piece_at<TI>(x.v[i][e / PE], e % PE), o[e], 0, 0, 0);
  };

  Tile A, B;
  constexpr int STEP = PT * PW;
  int t = t0 + w * PT;
  if (t < t1) load(A, t);
  while (t < t1) {
    if (t + STEP < t1) load(B, t + STEP);
    use(A);
    t += STEP;
    if (t >= t1) break;
    if (t + STEP < t1) load(A, t + STEP);
    use(B);
    t += STEP;
  }

  // the waves' parts, eight heads at a time
  l += __shfl_xor(l, 16);
  l += __shfl_xor(l, 32);
  if (g == 0) {
    sm[w][j] = m;
    sl[w][j] = l;
  }
  for (int hb = 0; hb < nh; hb += 8) {
    __syncthreads();
    if (g >> 1 == hb >> 3) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int c = 0; c < VP; ++c)
#pragma unroll
          for (int e = 0; e < PE; ++e) so[w][(4 * g + i) & 7][c * 16 * PE + j * PE + e] = o[c * PE + e][i];
    }
    __syncthreads();
    const int heads = nh - hb < 8 ? nh - hb : 8;
    for (int x = (int)threadIdx.x; x < heads * D; x += 64 * PW) {
      const int hh = x / D, d = x % D, h = hb + hh;
      float mx = sm[0][h];
#pragma unroll
      for (int u = 1; u < PW; ++u) mx = fmaxf(mx, sm[u][h]);
      float sum = 0.f, val = 0.f;
#pragma unroll
      for (int u = 0; u < PW; ++u) {
        const float f = sm[u][h] == kNone ? (sl[u][h] == 0.f ? 0.f : 1.f) : __builtin_amdgcn_exp2f(sm[u][h] - mx);
        sum += f * sl[u][h];
        val += f * so[u][hh][d];
      }
      const int64_t head = (int64_t)n * a.Hq + h0 + h;
      if constexpr (PART) {
        const int64_t at = head * splits + split;
        a.ws[at * D + d] = val;
        if (d == 0) {
          float* ml = a.ws + (int64_t)a.N * a.Hq * splits * D + at * 2;
          ml[0] = mx;
          ml[1] = sum;
        }
      } else {
        ((TI*)a.out)[(int64_t)n * a.out_rs + (int64_t)(h0 + h) * D + d] = (TI)(sum == 0.f ? 0.f : val / sum);
        if (d == 0 && a.lse) a.lse[head] = sum == 0.f ? kNone : (mx + log2f(sum)) * 0.69314718f;
      }
    }
  }
}

// Joins a head's chunks: one workgroup per (sequence, query head).
template <typename TI, int D> __global__ __launch_bounds__(256) void k_paged_join(PagedArgs a, int chunk, int splits) {
  constexpr int CG = D / 4, RG = 256 / CG;  // threads to a row of O, rows side by side
  __shared__ float red[8];
  __shared__ __align__(16) float acc[RG][D];
  const int n = (int)blockIdx.x / a.Hq;
  const PagedSpan sp = paged_span(a, n, chunk);
  const int64_t head = blockIdx.x;
  const float* O = a.ws + head * splits * D;
  const float* ml = a.ws + (int64_t)a.N * a.Hq * splits * D + head * splits * 2;
  float mx = kNone;
  for (int s = (int)threadIdx.x; s < sp.chunks; s += 256) mx = fmaxf(mx, ml[s * 2]);
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) mx = fmaxf(mx, __shfl_xor(mx, d));
  if (lane_id() == 0) red[wave_id()] = mx;
  __syncthreads();
  mx = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
  const int cg = (int)threadIdx.x % CG, rg = (int)threadIdx.x / CG;
  f32x4 val{0.f, 0.f, 0.f, 0.f};
  float sum = 0.f;
  for (int s = rg; s < sp.chunks; s += RG) {
    const float ms = ml[s * 2], ls = ml[s * 2 + 1];
    const float f = ms == kNone ? (ls == 0.f ? 0.f : 1.f) : __builtin_amdgcn_exp2f(ms - mx);
    sum += f * ls;
    val += f * *reinterpret_cast<const f32x4*>(O + (int64_t)s * D + cg * 4);
  }
  *reinterpret_cast<f32x4*>(&acc[rg][cg * 4]) = val;
  __shared__ float sums[RG];
  if (cg == 0) sums[rg] = sum;
  __syncthreads();
  if ((int)threadIdx.x < D) {
    float v = 0.f, t = 0.f;
#pragma unroll
    for (int i = 0; i < RG; ++i) {
      v += acc[i][threadIdx.x];
      t += sums[i];
    }
    ((TI*)a.out)[(int64_t)n * a.out_rs + (head - (int64_t)n * a.Hq) * D + threadIdx.x] = (TI)(t == 0.f ? 0.f : v / t);
    if (threadIdx.x == 0 && a.lse) a.lse[head] = t == 0.f ? kNone : (mx + log2f(t)) * 0.69314718f;
  }
}

// ------------------------------------------------------------------ launches
// Tokens per chunk: as many workgroups as fill the chip several times over, none with less than 256 tokens.
struct PagedPlan {
  int chunk, splits, gt;
};
static PagedPlan paged_plan(const PagedArgs& a) {
  PagedPlan p;
  const int r = a.Hq / a.Hk;
  p.gt = (r + 15) / 16;
  const int64_t span = (a.window > 0 && a.window < a.max_len ? a.window + PT - 1 : a.max_len);
  const int64_t rows = (int64_t)a.N * a.Hk * p.gt;
  int64_t want = rows ? (1024 + rows - 1) / rows : 1;
  int64_t chunk = (span + want - 1) / want;
  if (chunk < 256) chunk = 256;
  chunk = (chunk + PT * PW - 1) / (PT * PW) * (PT * PW);
  p.chunk = (int)(chunk < (1 << 30) ? chunk : 1 << 30);
  p.splits = (int)((span + p.chunk - 1) / p.chunk);
  if (p.splits < 1) p.splits = 1;
  return p;
}
size_t paged_ws_bytes(const PagedArgs& a, int) {
  const PagedPlan p = paged_plan(a);
  return p.splits == 1 ? 0 : (size_t)a.N * a.Hq * p.splits * (a.D + 2) * sizeof(float);
}

template <typename TI, int D, bool UNI> static hipError_t paged_go(const PagedArgs& a, hipStream_t s) {
  const PagedPlan p = paged_plan(a);
  const unsigned grid = (unsigned)((int64_t)a.N * a.Hk * p.gt * p.splits);
  traced("k_paged", s, [&] {
    if (p.splits == 1) k_paged<TI, D, UNI, false><<<grid, 64 * PW, 0, s>>>(a, p.chunk, 1, p.gt);
    else k_paged<TI, D, UNI, true><<<grid, 64 * PW, 0, s>>>(a, p.chunk, p.splits, p.gt);
  });
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.splits == 1) return e;
  traced("k_paged_join", s, [&] { k_paged_join<TI, D><<<(unsigned)((int64_t)a.N * a.Hq), 256, 0, s>>>(a, p.chunk, p.splits); });
  return hipGetLastError();
}
template <typename TI, int D> static hipError_t paged_uni(const PagedArgs& a, hipStream_t s) {
  return a.page % PT == 0 ? paged_go<TI, D, true>(a, s) : paged_go<TI, D, false>(a, s);
}
template <typename TI> static hipError_t paged_d(const PagedArgs& a, hipStream_t s) {
  switch (a.D) {
    case 32: return paged_uni<TI, 32>(a, s);
    case 64: return paged_uni<TI, 64>(a, s);
    case 128: return paged_uni<TI, 128>(a, s);
    case 256: return paged_uni<TI, 256>(a, s);
  }
  return hipErrorInvalidValue;
}
hipError_t launch_paged(const PagedArgs& a, int dtype, hipStream_t s) {
  if (a.N == 0) return hipSuccess;
  return dtype == 0 ? paged_d<float>(a, s) : paged_d<__bf16>(a, s);
}

}  // namespace gdn
