// paged_attn.hip -- attention of one new token per sequence over a paged cache, on gfx950.
//
//   z_t = scale q . k_t,  out = sum_t exp(z_t - lse) v_t,  lse = log sum_t exp(z_t)
//
// One pass over the cache with the running maximum m and sum l of the softmax, in log2 units. A workgroup takes a chunk of one
// sequence's tokens for up to 16 query heads of a key head, its waves tiles of 16 tokens in turn: every key and value is read once for
// each 16 query heads of its key head, and the kernel is bound by HBM (64 sequences of up to 8192 tokens, 4 key heads of 128, 16 query
// heads to each: bfloat16 120 us, float32 210; 17 to 32 of them, two reads: 216 to 228 and 388 to 408; 33: bfloat16 313).
// Nothing passes through LDS inside a tile:
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

// How a launch cuts its sequences into chunks, each a workgroup per key head and 16 query heads.
//   even: chunks of one length, found on the device from the lengths as they are, so that there are at most `slots`
//     of them (up to kPagedEven sequences); chunk c takes slot c of the workspace;
//   else: `chunk` tokens each, `splits` of them to every sequence, in use or not; slot n splits + split. Sequences of like lengths run
//     as fast (256 of up to 8000 tokens, 4 key heads of 128: 363 us, 257 365; of up to 1500 89 and 81), but a long one among short ones has
//     only its own few workgroups (one of 131072 among others of 200, 8 heads: 256 of them 185 us, 257 642).
constexpr int kPagedEven = 256;
struct PagedPlan {
  int gt, splits, slots, chunk;
  float share;  // even: chunks of up to 256 tokens are not below this part of all tokens
  bool even;
};

// What a sequence's length and window leave: tokens [lo, len), chunks from `base` on.
struct PagedSpan {
  int lo, len, base;
};
__device__ __forceinline__ PagedSpan paged_span(const PagedArgs& a, int n) {
  PagedSpan s;
  const int len = a.lens[n];
  s.len = len < 0 ? 0 : len > a.max_len ? a.max_len : len;
  s.lo = a.window > 0 && s.len > a.window ? s.len - a.window : 0;
  s.base = s.lo & ~(PT - 1);
  return s;
}

// Chunk `id` of a launch (ROWS = false), or the first chunk of sequence `id`: every sequence has one at least.
struct PagedChunk {
  int n, split, chunks, chunk, slot;
};
template <bool ROWS> __device__ __forceinline__ PagedChunk paged_chunk(const PagedArgs& a, const PagedPlan& p, int id) {
  PagedChunk c;
  if (!p.even) {
    c.n = ROWS ? id : id / p.splits;
    // turned from row to row, so that the launch's order (and with it an XCD) does not go with a chunk's number
    c.split = ROWS ? 0 : (id + c.n) % p.splits;
    c.chunk = p.chunk;
    const PagedSpan s = paged_span(a, c.n);
    c.chunks = s.len - s.base <= c.chunk ? 1 : (s.len - s.base + c.chunk - 1) / c.chunk;
    c.slot = c.n * p.splits + c.split;
    return c;
  }
  constexpr int U = kPagedEven / 64;  // lane l holds the sequences U l .. U l + U - 1
  int w[U];
  int64_t total = 0;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int n = lane_id() * U + u;
    w[u] = 0;
    if (n < a.N) {
      const PagedSpan s = paged_span(a, n);
      w[u] = s.len - s.base;
    }
    total += w[u];
  }
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) total += __shfl_xor(total, d);
  // at most total / chunk + N chunks
  int64_t want = (total + p.slots - a.N - 1) / (p.slots - a.N);
  const int round = (int)fminf((float)total * p.share, 256.f);
  want = want > round ? want : round;
  c.chunk = want <= p.chunk ? p.chunk : (int)((want + PT * PW - 1) / (PT * PW)) * (PT * PW);
  int cnt[U], sum = 0;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    cnt[u] = lane_id() * U + u >= a.N ? 0 : w[u] <= c.chunk ? 1 : (w[u] + c.chunk - 1) / c.chunk;
    sum += cnt[u];
  }
  int at = wave_scan_incl_int(sum) - sum, n = -1, split = 0, chunks = 0, slot = 0;  // chunks in front of this lane's
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const bool here = ROWS ? lane_id() * U + u == id : id >= at && id < at + cnt[u];
    if (here) {
      n = lane_id() * U + u;
      split = ROWS ? 0 : id - at;
      chunks = cnt[u];
      slot = ROWS ? at : id;
    }
    at += cnt[u];
  }
  const uint64_t who = __ballot(n >= 0);
  c.n = -1;
  if (who == 0) return c;
  const int l = __builtin_ctzll(who);
  c.n = __builtin_amdgcn_readlane(n, l);
  c.split = __builtin_amdgcn_readlane(split, l);
  c.chunks = __builtin_amdgcn_readlane(chunks, l);
  c.slot = __builtin_amdgcn_readlane(slot, l);
  return c;
}

// A lane's pieces of one key (KP of 16 bytes) and of one value row (VP pieces of PE values: D / 16 of them).
template <typename TI, int D> struct PagedTile {
  static constexpr int KP = D / (64 / (int)sizeof(TI));
  static constexpr int VE = D / 16, PE = VE < 16 / (int)sizeof(TI) ? VE : 16 / (int)sizeof(TI), VP = VE / PE;
  typedef int32_t vpiece __attribute__((ext_vector_type(PE * (int)sizeof(TI) / 4)));
};
template <> struct PagedTile<__bf16, 32> {
  static constexpr int KP = 1, VE = 2, PE = 2, VP = 1;
  typedef int32_t vpiece;
};

// Value e of a piece as float32.
template <typename TI, typename P> __device__ __forceinline__ float piece_at(const P& p, int e) {
  uint32_t w;
  if constexpr (sizeof(P) == 4) w = (uint32_t)p;
  else w = (uint32_t)p[sizeof(TI) == 2 ? e / 2 : e];
  if constexpr (sizeof(TI) == 2) w = e & 1 ? w & 0xFFFF0000u : w << 16;
  return __uint_as_float(w);
}

// Workgroups per compute unit of k_paged, whose registers grow with a head's bytes.
constexpr int paged_resident(int head_bytes) { return head_bytes <= 256 ? 4 : head_bytes <= 512 ? 2 : 1; }

template <typename TI, int D, bool UNI>
__global__ __launch_bounds__(64 * PW, paged_resident(D * (int)sizeof(TI))) void k_paged(PagedArgs a, PagedPlan plan) {
  typedef PagedTile<TI, D> Tile;
  constexpr int KP = Tile::KP, VE = Tile::VE, PE = Tile::PE, VP = Tile::VP;
  __shared__ __align__(16) float so[PW][8][D];
  __shared__ float sm[PW][16], sl[PW][16];
  // heads run fastest: those of a page lie together
  int bx = (int)blockIdx.x;
  const int hk = bx % a.Hk;
  bx /= a.Hk;
  const int ht = bx % plan.gt;
  const PagedChunk ch = paged_chunk<false>(a, plan, bx / plan.gt);
  if (ch.n < 0 || ch.split >= ch.chunks) return;
  const int n = ch.n, r = a.Hq / a.Hk, h0 = hk * r + ht * 16, nh = r - ht * 16 < 16 ? r - ht * 16 : 16;
  const PagedSpan sp = paged_span(a, n);
  const int w = wave_id(), g = lane_id() >> 4, j = lane_id() & 15;
  const int t0 = sp.base + ch.split * ch.chunk, t1 = sp.len - t0 < ch.chunk ? sp.len : t0 + ch.chunk;
  const TI *kp = (const TI*)a.kp, *vp = (const TI*)a.vp;
  const int* table = a.table + (int64_t)n * a.max_pages;

  i32x4 q[KP];
#pragma unroll
  for (int p = 0; p < KP; ++p) {
    q[p] = i32x4{0, 0, 0, 0};
    if (j < nh) q[p] = *reinterpret_cast<const i32x4*>((const TI*)a.q + (int64_t)n * a.q_rs + (int64_t)(h0 + j) * D + (p * 64 + g * 16) / (int)sizeof(TI));
  }
  const float sc = a.scale * 1.44269504f, sc_lo = fmaf(a.scale, 1.44269504f, -sc) + a.scale * 1.92596299e-8f;
  f32x4 o[VE];
#pragma unroll
  for (int e = 0; e < VE; ++e) o[e] = f32x4{0.f, 0.f, 0.f, 0.f};
  float m = kNone, l = 0.f;  // of head j; l: this lane's tokens only

  // Where a tile's tokens are. UNI: a tile lies in one page, and `row` is that of its first token; else `row` is that of
  // token t + j. mask: bit i: token 4g + i counts; full: every token does (wave-uniform). Every load is issued, that of a token
  // which does not count at a place inside the pool: a load that a branch may skip would make each wait one for all loads.
  struct Place {
    uint32_t row, mask;
    bool full;
  };
  auto entry = [&](int t) -> int {  // of the page table
    int u = UNI ? t : t + j;
    u = u < sp.lo ? sp.lo : u < t1 ? u : t1 - 1;
    if constexpr (UNI) return __builtin_amdgcn_readfirstlane(table[(uint32_t)u / (uint32_t)a.page]);
    else return table[(uint32_t)u / (uint32_t)a.page];
  };
  auto place = [&](int t, int page) -> Place {
    Place x;
    const bool in = page >= 0 && page < a.n_pages;
    const uint32_t base = ((uint32_t)(in ? page : 0) * (uint32_t)a.Hk + (uint32_t)hk) * (uint32_t)a.page;
    if constexpr (UNI) {
      x.row = base + (uint32_t)t % (uint32_t)a.page;
      x.full = in && t >= sp.lo && t + PT <= t1;
      x.mask = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) x.mask |= in && t + 4 * g + i >= sp.lo && t + 4 * g + i < t1 ? 1u << i : 0u;
    } else {
      x.row = base + (uint32_t)(t + j) % (uint32_t)a.page;
      const uint64_t all = __ballot(in && t + j >= sp.lo && t + j < t1);
      x.full = all == ~0ull;
      x.mask = (uint32_t)(all >> (4 * g)) & 15;  // (lanes 0 .. 15 hold the tile's tokens)
    }
    return x;
  };
  i32x4 k[KP];
  typename Tile::vpiece v[4][VP];
  auto load_k = [&](const Place& x) {
    const TI* p = kp + (int64_t)(UNI ? x.row + j : x.row) * D;
#pragma unroll
    for (int c = 0; c < KP; ++c) k[c] = __builtin_nontemporal_load(reinterpret_cast<const i32x4*>(p + (c * 64 + g * 16) / (int)sizeof(TI)));
  };
  auto load_v = [&](const Place& x) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t row;
      if constexpr (UNI) row = x.row + 4 * g + i;
      else row = (uint32_t)__builtin_amdgcn_ds_bpermute((4 * g + i) << 2, (int)x.row);
      const TI* p = vp + (int64_t)row * D;
#pragma unroll
      for (int c = 0; c < VP; ++c)
        v[i][c] = __builtin_nontemporal_load(reinterpret_cast<const typename Tile::vpiece*>(p + c * 16 * PE + j * PE));
    }
  };
  auto score = [&]() {
    f32x4 s{0.f, 0.f, 0.f, 0.f};
    if constexpr (sizeof(TI) == 2) {
#pragma unroll
      for (int c = 0; c < KP; ++c)
        s = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, k[c]), __builtin_bit_cast(bf16x8, q[c]), s, 0, 0, 0);
    } else {
      // four sums side by side: one chain of D products rounds twice as far (heads of 256: 1.1e-6 off the result in all, so 3.6e-7)
      f32x4 part[4] = {s, s, s, s};
#pragma unroll
      for (int c = 0; c < KP; ++c)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          part[e] = __builtin_amdgcn_mfma_f32_16x16x4f32(__int_as_float(k[c][e]), __int_as_float(q[c][e]), part[e], 0, 0, 0);
      s = (part[0] + part[1]) + (part[2] + part[3]);
    }
    return s;
  };
  auto add = [&](const f32x4& s, const Place& x) {
    float z[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) z[i] = x.full || x.mask >> i & 1 ? s[i] * sc : kNone;
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
      // (float32: the score times sc in two parts, without the product's rounding)
      if constexpr (sizeof(TI) == 4) p[i] = z[i] == kNone ? 0.f : __builtin_amdgcn_exp2f(fmaf(s[i], sc, fmaf(s[i], sc_lo, -ref)));
      else p[i] = __builtin_amdgcn_exp2f(z[i] - ref);
      l += p[i];
    }
    if (!x.full)  // what lies in a place that does not count may be anything, NaN too
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int c = 0; c < VP; ++c) v[i][c] = x.mask >> i & 1 ? v[i][c] : typename Tile::vpiece{};
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int e = 0; e < VE; ++e)
        o[e] = __builtin_amdgcn_mfma_f32_16x16x4f32(p[i], piece_at<TI>(v[i][e / PE], e % PE), o[e], 0, 0, 0);
  };

  constexpr int STEP = PT * PW;
  int t = t0 + w * PT;
  if (t < t1 && a.n_pages > 0) {
    int e1 = entry(t + STEP);
    Place at = place(t, entry(t));
    load_k(at);
    load_v(at);
    for (; t + STEP < t1; t += STEP) {
      const f32x4 s = score();
      __builtin_amdgcn_sched_barrier(0);  // (loads moved up would need registers of their own, and spill)
      // the keys are used up: the next tile's take their registers while this one's weights and values are worked on
      const Place next = place(t + STEP, e1);
      e1 = entry(t + 2 * STEP);
      load_k(next);
      __builtin_amdgcn_sched_barrier(0);
      add(s, at);
      __builtin_amdgcn_sched_barrier(0);
      load_v(next);
      __builtin_amdgcn_sched_barrier(0);
      at = next;
    }
    add(score(), at);
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
        const float f = sm[u][h] == kNone ? 1.f : __builtin_amdgcn_exp2f(sm[u][h] - mx);  // (of none: no sum, or a NaN)
        sum += f * sl[u][h];
        val += f * so[u][hh][d];
      }
      const int64_t head = (int64_t)n * a.Hq + h0 + h;
      if (ch.chunks > 1) {
        const int64_t at = (int64_t)ch.slot * a.Hq + h0 + h;
        a.ws[at * D + d] = val;
        if (d == 0) {
          float* ml = a.ws + (int64_t)plan.slots * a.Hq * D + at * 2;
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

// Joins the chunks of HB heads of a sequence, 64 columns of each (JC): SG groups of threads take every SG-th chunk, with a
// running maximum of their own.
template <typename TI, int D, int SG> __global__ __launch_bounds__(256) void k_paged_join(PagedArgs a, PagedPlan plan) {
  constexpr int JC = D < 64 ? D : 64, CG = JC / 4, HB = 256 / CG / SG;
  __shared__ float sm[SG][HB], sl[SG][HB];
  __shared__ __align__(16) float acc[SG][HB][JC];
  const int hblocks = (a.Hq + HB - 1) / HB, n = (int)blockIdx.x / hblocks, c0 = (int)blockIdx.y * JC;
  const PagedChunk ch = paged_chunk<true>(a, plan, n);
  if (ch.chunks == 1) return;
  const int cg = (int)threadIdx.x % CG, unit = (int)threadIdx.x / CG, sg = unit % SG, hb = unit / SG;
  const int h = ((int)blockIdx.x - n * hblocks) * HB + hb;
  float m = kNone, l = 0.f;
  f32x4 val{0.f, 0.f, 0.f, 0.f};
  if (h < a.Hq) {
    const float* O = a.ws + ((int64_t)ch.slot * a.Hq + h) * D + c0 + cg * 4;
    const float* ml = a.ws + (int64_t)plan.slots * a.Hq * D + ((int64_t)ch.slot * a.Hq + h) * 2;
#pragma unroll 4
    for (int s = sg; s < ch.chunks; s += SG) {
      const float ms = ml[(int64_t)s * a.Hq * 2], ls = ml[(int64_t)s * a.Hq * 2 + 1];
      const f32x4 os = *reinterpret_cast<const f32x4*>(O + (int64_t)s * a.Hq * D);
      const float mx = fmaxf(m, ms), f = m == kNone ? 0.f : __builtin_amdgcn_exp2f(m - mx);
      // (a chunk of which nothing is left has no sum, or a NaN)
      const float fs = ms == kNone ? 1.f : __builtin_amdgcn_exp2f(ms - mx);
      m = mx;
      l = l * f + fs * ls;
      val = val * f + fs * os;
    }
  }
  *reinterpret_cast<f32x4*>(&acc[sg][hb][cg * 4]) = val;
  if (cg == 0) {
    sm[sg][hb] = m;
    sl[sg][hb] = l;
  }
  __syncthreads();
  for (int x = (int)threadIdx.x; x < HB * JC; x += 256) {
    const int hh = x / JC, c = x % JC, head = ((int)blockIdx.x - n * hblocks) * HB + hh;
    if (head >= a.Hq) continue;
    float mx = sm[0][hh], v = 0.f, t = 0.f;
#pragma unroll
    for (int i = 1; i < SG; ++i) mx = fmaxf(mx, sm[i][hh]);
#pragma unroll
    for (int i = 0; i < SG; ++i) {
      const float f = sm[i][hh] == kNone ? 1.f : __builtin_amdgcn_exp2f(sm[i][hh] - mx);
      t += f * sl[i][hh];
      v += f * acc[i][hh][c];
    }
    ((TI*)a.out)[(int64_t)n * a.out_rs + (int64_t)head * D + c0 + c] = (TI)(t == 0.f ? 0.f : v / t);
    if (c0 + c == 0 && a.lse) a.lse[(int64_t)n * a.Hq + head] = t == 0.f ? kNone : (mx + log2f(t)) * 0.69314718f;
  }
}

// ------------------------------------------------------------------ launches
// Chunks: as many as the chip holds workgroups at once, so that equal ones end together (one sequence of 131072 tokens, 4 heads
// of 256: 93 us with 512 of them, 99 with 1024, 114 with 2048), and four more for every sequence, whose last chunks are
// of unequal lengths (64 sequences of up to 8192 tokens, 8 heads of 128: 217 us with 1024, 195 with 2048, 190 with
// 4096), but of less than 256 tokens no more than the chip holds (32 sequences of 1000 tokens, 8 heads of 128: 34 us, with four more 38;
// 128 of up to 1500, 4 heads: 51 and 56). None of less than 128 tokens, two tiles for each wave. A launch for the join is not worth it for a few tiles more: up to
// 512 tokens (256 of heads past 256 bytes) are one chunk (64 sequences of up to 500 tokens, 8 heads of 128: 23 us, with a join 26; 16
// of 300, heads of 64: 12 and 17; one of 500: 14 and 17; but one of 1000 24 and 17, 9 of 500, heads of 256: 25 and 17).
static PagedPlan paged_plan(const PagedArgs& a, int dtype) {
  PagedPlan p;
  p.gt = (a.Hq / a.Hk + 15) / 16;
  p.share = 0.f;
  const int64_t span = a.window > 0 && a.window < a.max_len ? (int64_t)a.window + PT - 1 : a.max_len;
  const int head_bytes = a.D * (dtype == 0 ? 4 : 2);
  const int64_t heads = (int64_t)a.Hk * p.gt, full = 256 * paged_resident(head_bytes), one = head_bytes <= 256 ? 512 : 256;
  const int64_t want = (full + heads - 1) / heads + 4 * (int64_t)a.N;
  constexpr int least = 128;
  p.even = a.N <= kPagedEven && span > one;
  if (p.even) {
    const int64_t most = a.N * ((span + least - 1) / least);
    p.chunk = least;
    p.splits = 0;
    p.share = (float)heads / (float)full;
    p.slots = (int)(want < most ? want : most) + a.N;
  } else {
    const int64_t each = (want + a.N - 1) / (a.N > 0 ? a.N : 1);
    int64_t chunk = span <= one ? span : (span + each - 1) / each;
    chunk = chunk < least ? least : (chunk + PT * PW - 1) / (PT * PW) * (PT * PW);
    p.chunk = (int)(chunk < (1 << 30) ? chunk : 1 << 30);
    p.splits = span > 0 ? (int)((span + p.chunk - 1) / p.chunk) : 1;
    p.slots = a.N * p.splits;
  }
  return p;
}
int64_t paged_blocks(const PagedArgs& a, int dtype) {
  const PagedPlan p = paged_plan(a, dtype);
  return (int64_t)p.slots * a.Hk * p.gt;
}
size_t paged_ws_bytes(const PagedArgs& a, int dtype) {
  const PagedPlan p = paged_plan(a, dtype);
  return p.splits == 1 ? 0 : (size_t)p.slots * a.Hq * (a.D + 2) * sizeof(float);
}

template <typename TI, int D, bool UNI> static hipError_t paged_go(const PagedArgs& a, hipStream_t s) {
  constexpr int dtype = sizeof(TI) == 2;
  const PagedPlan p = paged_plan(a, dtype);
  const unsigned grid = (unsigned)paged_blocks(a, dtype);
  traced("k_paged", s, [&] { k_paged<TI, D, UNI><<<grid, 64 * PW, 0, s>>>(a, p); });
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.splits == 1) return e;
  // few sequences may have many chunks each, many have few
  constexpr int units = D < 64 ? 32 : 16;
  const unsigned cols = D < 64 ? 1 : D / 64;
  traced("k_paged_join", s, [&] {
    if ((int64_t)a.N * a.Hq * cols <= 512) k_paged_join<TI, D, units><<<dim3((unsigned)(a.N * a.Hq), cols), 256, 0, s>>>(a, p);
    else k_paged_join<TI, D, 2><<<dim3((unsigned)(a.N * ((a.Hq + units / 2 - 1) / (units / 2))), cols), 256, 0, s>>>(a, p);
  });
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
